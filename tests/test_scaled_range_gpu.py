"""Scaled products whose scales are far from 1, up to the ends of the range that is promised: the two
scales that meet, and a group's sum with either of them, have a product that is a normal
number of fp32 (or zero)."""
import pytest
import torch

from persistent_stream_matmul_gb300 import _binding as B
from scaled_util import assert_product, quantized
from test_scaled_gpu import BLOCK, COL, ROW, VEC, Case

pytestmark = pytest.mark.gpu

FORMS = [(1, B.GEMM_SCALED_FEW), (1, B.GEMM_SCALED_STRAIGHT), (2, B.GEMM_SCALED_STRAIGHT), (1, B.GEMM_SCALED_TURNED)]
# (of A, of B), as powers of two; the scales are that times exp of a normal value, 2^-7 to 2^7
RANGES = [(-100, -10), (-10, -100), (-55, -55), (80, 15), (15, 80), (50, 45), (-100, 80), (80, -100)]


@pytest.fixture(scope="module", autouse=True)
def _ready():
    from gpu_util import ensure_built
    ensure_built()


@pytest.mark.parametrize("ctas,form", FORMS)
@pytest.mark.parametrize("scale_a,scale_b", [(VEC, BLOCK), (VEC, VEC), (BLOCK, BLOCK)])
@pytest.mark.parametrize("pa,pb", RANGES)
@pytest.mark.parametrize("layout_b", [COL, ROW])
def test_scales_far_from_one(pa, pb, layout_b, scale_a, scale_b, ctas, form):
    """Sums of a group of positive values are near 128 * 64 * 64 = 2^19, so each product on the way is between 2^-124
    and 2^128 / 2."""
    if form == B.GEMM_SCALED_FEW and layout_b == ROW:
        pytest.skip("the form needs contiguous sums")
    c = Case(40, 272, 400, a="e5m2", out="f32", layout_b=layout_b, scale_a=scale_a, scale_b=scale_b, seed=pa - pb + 300, ctas=ctas, form=form)
    for t in (c.a, c.b):
        t.copy_((t.float().abs() + 1).to(t.dtype))
    c.sa *= 2.0 ** pa
    c.sb *= 2.0 ** pb
    exact, absolute = c.reference()
    assert_product(c.run(), exact, absolute, c.K)


@pytest.mark.parametrize("ctas,form", FORMS)
@pytest.mark.parametrize("scale_b", [VEC, BLOCK])
def test_groups_of_zeros_and_of_tiny_values(scale_b, ctas, form):
    """Rows and blocks as the quantisation makes them of zeros and of values of 2^-70: scales down to 2^-109, and
    products of them that vanish.  Every part of the result is within 2^-125 (three groups)."""
    c = Case(33, 272, 272, out="f32", scale_b=scale_b, ctas=ctas, form=form)
    for t, s, kind in ((c.a, c.sa, c.kinds[0]), (c.b, c.sb, c.kinds[1])):
        x = t.float() / 448
        x[5:30] *= 2.0 ** -70
        x[:4] = 0
        x[:, 130:] = 0 if kind == "blocks" else 2.0 ** -70 * x[:, 130:]
        q, sc = quantized(x.double(), "e4m3", kind)
        t.copy_(q.float().to(t.dtype))
        s.copy_(sc.float())
    exact, absolute = c.reference()
    got = c.run()
    assert bool(torch.isfinite(got).all())
    got = torch.where((got.double() - exact).abs() <= 3 * 2.0 ** -125, exact.float(), got)
    assert_product(got, exact, absolute, c.K)
