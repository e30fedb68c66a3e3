"""Scaled products that are bound by the store of C: many tiles a scheduling unit, one to three
k-blocks each, so that a tile is staged while the copies of the one before are still on
their way.  Whole numbers, compared bit for bit."""
import pytest
import torch

from persistent_stream_matmul_gb300 import _binding as B
from test_scaled_gpu import BLOCK, COL, ROW, VEC, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    from gpu_util import ensure_built
    ensure_built()


@pytest.mark.parametrize("K", [16, 128, 272, 384])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("layouts,scale_b", [((ROW, COL), BLOCK), ((COL, ROW), VEC)], ids=["forward", "gradient"])
def test_tiles_in_quick_succession(layouts, scale_b, ctas, out, K):
    """Boxes a tile and warp: 2 (one CTA, 16 bits), 4 (one CTA fp32, pairs 16 bits) or 8 (pairs, fp32)."""
    c = Case(5120, 6144, K, out=out, layout_a=layouts[0], layout_b=layouts[1], scale_b=scale_b, integers=True, seed=K, form=B.GEMM_SCALED_STRAIGHT,
             ctas=ctas)
    assert c.plan.info("tiles") > 6 * c.plan.info("units")
    # whole sixteenths below 9 * 16 * 384 < 2^16: exact in fp32 in any order, rounded once
    want = c.reference()[0].float().to(c.dtype)
    for _ in range(6):
        assert torch.equal(c.run(), want)
