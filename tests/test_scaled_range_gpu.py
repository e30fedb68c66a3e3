"""Scaled products whose scales are far from 1: the two scales that meet may have a
product outside the normal range of fp32 where the result is inside it."""
import pytest
import torch

from persistent_stream_matmul_gb300 import _binding as B
from scaled_util import assert_product
from test_scaled_gpu import COL, ROW, VEC, BLOCK, Case

pytestmark = pytest.mark.gpu

FORMS = [(1, B.GEMM_SCALED_FEW), (1, B.GEMM_SCALED_STRAIGHT), (2, B.GEMM_SCALED_STRAIGHT), (1, B.GEMM_SCALED_TURNED)]
# (of A, of B), as powers of two
RANGES = [(-113, -37), (-37, -113), (-109, -19), (-75, -75), (-100, -40), (80, 60), (-100, 80), (80, -100)]


@pytest.fixture(scope="module", autouse=True)
def _ready():
    from gpu_util import ensure_built
    ensure_built()


@pytest.mark.parametrize("ctas,form", FORMS)
@pytest.mark.parametrize("scale_a,scale_b", [(VEC, BLOCK), (VEC, VEC), (BLOCK, BLOCK)])
@pytest.mark.parametrize("pa,pb", RANGES)
@pytest.mark.parametrize("layout_b", [COL, ROW])
def test_scales_far_from_one(pa, pb, layout_b, scale_a, scale_b, ctas, form):
    """Sums of a group are near 128 * 100^2 = 2^20, and none is small: fp32 output is within the bound of any other
    product wherever it is a normal number.  Where it is not (2^20 * 2^-150), it is within a few of its smallest steps;
    where it is past the largest (2^20 * 2^140), infinite."""
    if form == B.GEMM_SCALED_FEW and layout_b == ROW:
        pytest.skip("the form needs contiguous sums")
    c = Case(40, 272, 400, a="e5m2", out="f32", layout_b=layout_b, scale_a=scale_a, scale_b=scale_b, seed=pa - pb + 300, ctas=ctas, form=form)
    # positive values, so that no sum is small by chance
    for t in (c.a, c.b):
        t.copy_(((t.float() * 2).abs() + 1).to(t.dtype))
    c.sa *= 2.0 ** pa
    c.sb *= 2.0 ** pb
    exact, absolute = c.reference()
    got = c.run()
    over = exact > 2.0 ** 129  # far past it
    assert bool(torch.isinf(got[over]).all())
    # (a subnormal sum of four groups: half a smallest step for each of two products and the addition)
    slack = 4 * 3 * 2.0 ** -150
    got = torch.where((got.double() - exact).abs() <= slack, exact.float(), got)
    assert_product(got, exact, absolute, c.K)


@pytest.mark.parametrize("ctas,form", FORMS)
@pytest.mark.parametrize("scale_b", [VEC, BLOCK])
def test_large_scales_of_zeros(scale_b, ctas, form):
    """Scales whose product overflows, over sums of nothing but zeros: the result is zero."""
    c = Case(33, 272, 272, out="f32", scale_b=scale_b, ctas=ctas, form=form)
    c.a.copy_(torch.zeros_like(c.a.float()).to(c.a.dtype))
    c.sa.fill_(2.0 ** 80)
    c.sb.fill_(2.0 ** 80)
    assert not c.run().any()
