"""Quantisation of every pair of mantissas: each of a 16-bit type's against each as the largest of its
group, where quotients lie on the borders between 8-bit values most often."""
import pytest
import torch

from moe_util import Rows
from scaled_util import DTYPES
from test_scaled_rows_gpu import check_quantized

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    from gpu_util import ensure_built
    ensure_built()


def pairs(bits, power):
    """(mantissas, elements): row i has the largest 2^bits + i at the start of every group of 128, and every mantissa
    times 2^power below it, in turn over the groups; signs alternate."""
    n = 2 ** bits
    groups = -(-n // 127)
    x = torch.arange(groups * 127, device="cuda") % n + n
    x = x * (1 - 2 * (torch.arange(groups * 127, device="cuda") % 2))
    rows = torch.empty(n, groups, 128, dtype=torch.float64, device="cuda")
    rows[:, :, 0] = (torch.arange(n, device="cuda") + n)[:, None]
    rows[:, :, 1:] = x.view(groups, 127) * 2.0 ** power
    return rows.view(n, groups * 128)


# x / m from 1 down to where the 8-bit values have no leading one, and vanish (e4m3: 2^-15 to 2^-19; e5m2: 2^-30 to
# 2^-33, which fp16 does not reach)
POWERS = {"bf16": (-1, -2, -9, -15, -16, -17, -18, -19, -29, -30, -31, -32, -33), "f16": (-1, -2, -9, -14, -15, -16, -17, -18, -19)}


@pytest.mark.parametrize("kind", ["rows", "cols", "blocks", "both"])
@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype,bits", [("bf16", 7), ("f16", 10)])
def test_every_pair(dtype, bits, type, kind):
    dt = DTYPES[dtype][1]
    for power in POWERS[dtype]:
        x = pairs(bits, power)
        n, cols = x.shape
        if kind == "cols":
            x = x.t().contiguous()
        elif kind == "blocks":
            # a block a row of the table: its elements, then zeros
            x = torch.nn.functional.pad(x, (0, 128 * 128 - cols)).view(n, 128, 128)
            side = 32 if bits == 10 else 8
            x = x.view(n // side, side, 128, 128).permute(0, 2, 1, 3).reshape(n // side * 128, side * 128)
        x16 = x.to(dt)
        assert torch.equal(x16.double(), x)  # the type holds every one
        check_quantized(Rows(*x.shape, dt).set(x16), type, kind)
