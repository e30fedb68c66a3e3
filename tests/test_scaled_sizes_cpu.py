"""Sizes of the 8-bit linear layer's workspaces at their least.  A child process asks, so that one
that dies shows as a failure."""
import subprocess
import sys

import pytest

from persistent_stream_matmul_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("rows,hidden,bytes", [(0, 0, 0), (0, 16, 0), (4, 0, 0), (2 ** 31 - 1024, 0, 0), (1, 1, 4), (4, 16, 256), (1, 32768, 131072)])
def test_norm_grad_workspace(rows, hidden, bytes):
    """A block a row at most, and a sum of hidden fp32 values a block."""
    code = ("from persistent_stream_matmul_gb300 import _binding as B\n"
            "print(B.gemm_rms_norm_grad_workspace_size(%d, %d))" % (rows, hidden))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)
    assert int(r.stdout) == bytes
