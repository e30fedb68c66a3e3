"""The 8-bit output of the root-mean-square norm, value for value.

y / m is z / (the largest |z| of the group) for z = s * weight: the row's factor
cancels.  z has at most 22 bits, so it and 448 z are exact in 64 bits; a quotient that
lies on a border between two 8-bit values has 5 bits, so the division gives it
exactly, and one that does not is 2^-27 of it away at least, 2^25 times the
division's rounding.  So the nearest 8-bit value is known for every element."""
import pytest
import torch

from moe_util import Rows
from persistent_stream_matmul_gb300 import _binding as B
from scaled_util import DTYPES, FP8, activations, quantized, scale_shape

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    from gpu_util import ensure_built
    ensure_built()


def run(x, w, type, residual=None, eps=1e-5, ldq=None, offset=0):
    """(values, scales, rstd) of the norm of x + residual."""
    rows, H = x.shape
    code = {torch.bfloat16: B.GEMM_BF16, torch.float16: B.GEMM_F16}[x.dtype]
    q = Rows(rows, H, torch.uint8, ldq, offset)
    scales, rstd = Rows(*scale_shape("rows", rows, H), torch.float32), torch.empty(rows, device="cuda")
    s = None if residual is None else torch.empty_like(x)
    B.gemm_rms_norm(x, H, residual, H, w, eps, rows, H, code, s, H, None, 0, q, q.ld, FP8[type][0], scales, rstd)
    q.check_guards()
    scales.check_guards()
    return q.view.contiguous().view(FP8[type][1]).double(), scales.view, rstd


def check(x, w, type, residual=None, **kw):
    got, scales, rstd = run(x, w, type, residual, **kw)
    s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    z = s.double() * w.double()
    want, m = quantized(z, type, "rows")
    assert torch.equal(got, want), "%d values" % int((got != want).sum())
    # m's product with the row's factor and the division round, 2^-24 each
    exact = m * rstd.double()
    assert bool(((scales.double() - exact).abs() <= 2 * 1.01 * 2.0 ** -24 * exact).all())


SIZES = [(1, 4096), (300, 4096), (64, 128), (37, 130), (5, 250), (200, 2056), (100, 5001), (40, 8200), (6, 20011), (3, 32768)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,H", SIZES)
def test_values_of_a_network(rows, H, dtype, type, residual):
    dt = DTYPES[dtype][1]
    x = activations((rows, H), dt, rows + H, 0.7)
    r = activations((rows, H), dt, rows + H + 1, 0.0) if residual else None
    w = (1 + 0.2 * torch.randn(H, generator=torch.Generator(device="cuda").manual_seed(H), device="cuda")).to(dt)
    check(x, w, type, r)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,H", [(256, 1024), (100, 1001), (8, 17000)])
@pytest.mark.parametrize("ldq,offset", [(0, 0), (3, 1)])
def test_borders_are_common(rows, H, dtype, type, ldq, offset):
    """Small whole numbers times powers of two: a large share of the quotients lie on a border, also
    where the 8-bit value has no leading one."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    dt = DTYPES[dtype][1]
    x = torch.randint(-31, 32, (rows, H), generator=g, device="cuda").float()
    x = (x * torch.exp2(torch.randint(-12, 1, (rows, H), generator=g, device="cuda").float())).to(dt)
    w = (torch.randint(1, 8, (H,), generator=g, device="cuda").float() / 8).to(dt)
    x[:, ::128] = 28.0  # 448 and 57344 are 28 times a power of two: the group's largest is often 28 * 7 / 8 or so
    w[::128] = 1.0
    check(x, w, type, ldq=H + ldq, offset=offset)


@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
def test_factors_of_one(type):
    """Rows of +-1 and eps 0: rstd is 1, so y is the weight and is known exactly, also where s * weight is
    small or below the least that a scale is made from."""
    H = 512
    x = torch.where(torch.rand(64, H, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") < 0.5, 1.0, -1.0).bfloat16()
    for power in (0, 60, 120, -70, -79, -81, -90, -99, -100, -101, -110, -126):
        w = activations((1, H), torch.bfloat16, power + 200, 0.0)[0] * 2.0 ** power
        got, scales, rstd = run(x, w, type, eps=0.0)
        assert bool((rstd == 1).all())
        want, m = quantized(x.double() * w.double(), type, "rows")
        assert torch.equal(got, want) and torch.equal(scales, m.float())


@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
def test_products_near_the_ends_of_the_range(type):
    """Rows of +-2^a have rstd 2^-a, so y is the weight; s * weight is a power of two of it, in fp32's range as
    long as it is above 2^-120 and below 2^127.  Past that the group counts as infinite."""
    H = 384
    sign = torch.where(torch.rand(32, H, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") < 0.5, 1.0, -1.0)
    for a, power in ((40, 80), (59, 60), (-60, -50), (-50, -60), (-60, 0), (59, -60), (0, -115), (30, -130)):
        x = (sign * 2.0 ** a).bfloat16()
        w = activations((1, H), torch.bfloat16, 3, 0.0)[0] * 2.0 ** power
        got, scales, rstd = run(x, w, type, eps=0.0)
        assert bool((rstd == 2.0 ** -a).all())
        want, m = quantized(sign.double() * w.double(), type, "rows")
        assert torch.equal(got, want) and torch.equal(scales, m.float())
    w = activations((1, H), torch.bfloat16, 3, 0.0)[0] * 2.0 ** 100
    got, scales, _ = run((sign * 2.0 ** 40).bfloat16(), w, type, eps=0.0)
    assert bool(torch.isinf(scales).all()) and bool(torch.isnan(got * scales.t().repeat_interleave(128, 1)).all())


def test_nan_infinity_and_zeros():
    """A NaN of the weight is its column's alone, one of a row the row's; a group with an infinite y stands
    for NaN; rows of zeros are zeros, with eps 0 NaN."""
    H = 256
    x = activations((6, H), torch.bfloat16, 4, 0.0)
    x[1] = 0
    x[2, 5] = float("nan")
    w = torch.ones(H, device="cuda").bfloat16()
    w[200] = float("nan")
    got, scales, _ = run(x, w, "e4m3")
    bad = torch.zeros(6, H, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 200] = True, True
    assert torch.equal(torch.isnan(got), bad)
    good = w.clone()
    good[200] = 0
    x[2] = 0
    want, _ = quantized(x.double() * good.double(), "e4m3", "rows")
    assert torch.equal(got[~bad], want[~bad]) and bool(torch.isfinite(scales).all())
    w = torch.ones(H, device="cuda").bfloat16()
    w[3] = float("inf")
    got, scales, _ = run(x, w, "e4m3")
    keep = [0, 3, 4, 5]
    assert bool(torch.isinf(scales[0, keep]).all()) and bool(torch.isfinite(scales[1]).all())
    assert bool(torch.isnan(got[:, :128] * scales[0].double()[:, None])[keep].all()) and bool(torch.isfinite(got[:, 128:]).all())
    got, scales, _ = run(x, torch.ones(H, device="cuda").bfloat16(), "e4m3", eps=0.0)
    assert torch.equal(torch.isnan(got).all(1), torch.isnan(got).any(1))
    assert torch.isnan(got).any(1).tolist() == [False, True, True, False, False, False]


@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
def test_quotients_next_to_a_border(type):
    """fp16: s is chosen for each element so that s * weight * L / m is as near to a border as it gets without being
    on it; dozens are within half of fp32's last digit of one."""
    rows, H = 512, 1024
    g = torch.Generator(device="cuda").manual_seed(7)
    w = torch.randint(1024, 2048, (H,), generator=g, device="cuda").double()
    top = torch.randint(1024, 2048, (rows, H // 128), generator=g, device="cuda").double()
    m = (top * w[::128]).repeat_interleave(128, 1)                    # of each element's group
    digits = 4 if type == "e4m3" else 3
    best, near = torch.full((rows, H), 1024.0, dtype=torch.float64, device="cuda"), torch.ones(rows, H, dtype=torch.float64, device="cuda")
    for t in range(2 ** digits + 1, 2 ** (digits + 1), 2):           # 1.xxx1 times a power of two
        s = t * m / (7 * w)
        s = s * torch.exp2(10 - torch.floor(torch.log2(s)))           # 11 bits before the point
        r = torch.round(s)
        d = (r - s).abs() / s
        ok = (d > 2.0 ** -40) & (d < near) & (r < 2048)
        best, near = torch.where(ok, r, best), torch.where(ok, d, near)
    assert int((near < 2.0 ** -25).sum()) > 10
    x = best / 4
    x[:, ::128] = top
    check(x.half(), (w / 1024).half(), type)
