"""Quantisation and the root-mean-square norm with its gradient against their
definitions in 64 bits."""
import pytest
import torch

from moe_util import Rows
from persistent_stream_matmul_gb300 import _binding as B
from scaled_util import DTYPES, FP8, KINDS, ROUNDOFF, activations, magnitudes, quantized, scale_shape, spread, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    from gpu_util import ensure_built
    ensure_built()


class Values(Rows):
    """An 8-bit matrix with guards, as bytes; the view as its type."""

    def __init__(self, rows, cols, type, ld=None, offset=0):
        super().__init__(rows, cols, torch.uint8, ld, offset)
        self.type = FP8[type][1]

    def values(self):
        return self.view.contiguous().view(self.type).double()


def table(shape):
    return Rows(*shape, torch.float32)


def quantize(x, type, kind, ldq=None, offset=0):
    rows, cols = x.rows, x.cols
    code = {torch.bfloat16: B.GEMM_BF16, torch.float16: B.GEMM_F16}[x.view.dtype]
    if kind == "both":
        out = [(Values(rows, cols, type, ldq, offset), table(scale_shape(k, rows, cols))) for k in ("rows", "cols")]
        (q0, s0), (q1, s1) = out
        B.gemm_scaled_quantize_both(x, x.ld, rows, cols, code, FP8[type][0], q0, q0.ld, s0, q1, q1.ld, s1)
    else:
        out = [(Values(rows, cols, type, ldq, offset), table(scale_shape(kind, rows, cols)))]
        q, s = out[0]
        B.gemm_scaled_quantize(KINDS[kind], x, x.ld, rows, cols, code, FP8[type][0], q, q.ld, s)
    for q, s in out:
        q.check_guards()
        s.check_guards()
    return out


def check_quantized(x, type, kind, **kw):
    got = quantize(x, type, kind, **kw)
    for (q, s), k in zip(got, ("rows", "cols") if kind == "both" else (kind,)):
        want, scales = quantized(x.view.double(), type, k)
        assert torch.equal(q.values(), want), k
        assert torch.equal(s.view, scales.float()), k  # one rounding


SIZES = [(1, 1), (1, 128), (1, 14336), (2, 127), (3, 129), (7, 16), (8, 200), (9, 1024), (127, 130), (128, 128), (129, 257),
         (300, 264), (1000, 1), (513, 2056)]


@pytest.mark.parametrize("kind", ["rows", "cols", "blocks", "both"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize(kind, dtype, type, rows, cols):
    x = Rows(rows, cols, DTYPES[dtype][1]).set(activations((rows, cols), DTYPES[dtype][1], rows * 7 + cols))
    check_quantized(x, type, kind)


@pytest.mark.parametrize("kind", ["rows", "cols", "blocks", "both"])
@pytest.mark.parametrize("ldx,off,ldq,offq", [(272, 0, 264, 0), (272, 8, 272, 8), (265, 0, 264, 0), (264, 1, 264, 0), (264, 3, 269, 5),
                                              (264, 0, 264, 4)])
def test_quantize_strides(kind, ldx, off, ldq, offq):
    x = Rows(140, 264, torch.bfloat16, ldx, off).set(activations((140, 264), torch.bfloat16, 5))
    check_quantized(x, "e4m3", kind, ldq=ldq, offset=offq)


@pytest.mark.parametrize("kind", ["rows", "cols", "blocks", "both"])
@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
def test_quantize_every_pair_of_mantissas(kind, type):
    """Quotients of 16-bit values often lie on a border between two 8-bit ones: every 11-bit
    mantissa of x against the largest of its group, over a range of the latter."""
    x = torch.rand(256, 256, device="cuda") * 0 + 1
    g = torch.Generator(device="cuda").manual_seed(11)
    for _ in range(4):
        x = (torch.randint(1024, 2048, (256, 256), generator=g, device="cuda").float() / 1024
             * torch.exp2(torch.randint(-18, 1, (256, 256), generator=g, device="cuda").float()))
        x = x * torch.sign(torch.randn(256, 256, generator=g, device="cuda"))
        check_quantized(Rows(256, 256, torch.float16).set(x), type, kind)
        check_quantized(Rows(256, 256, torch.bfloat16).set(x), type, kind)


@pytest.mark.parametrize("kind", ["rows", "cols", "blocks", "both"])
def test_quantize_extremes(kind):
    x = torch.zeros(256, 256, device="cuda")
    x[128:] = 3e38  # bf16's largest values, beside zeros and its smallest
    x[:128, 128:] = 1e-40
    x[5, 7] = -2.0 ** -133
    rows = Rows(256, 256, torch.bfloat16).set(x)
    for type in FP8:
        check_quantized(rows, type, kind)


@pytest.mark.parametrize("kind", ["rows", "cols", "blocks"])
def test_quantize_nan_and_infinity(kind):
    x = activations((256, 256), torch.bfloat16, 3)
    x[3, 5], x[200, 130] = float("nan"), float("-inf")
    (q, s), = quantize(Rows(256, 256, torch.bfloat16).set(x), "e4m3", kind)
    m = magnitudes(x.double(), kind)
    assert torch.equal(torch.isinf(s.view), torch.isinf(m))
    stands_for = q.values() * spread(s.view.double(), 256, 256, kind)
    bad = torch.isinf(spread(m, 256, 256, kind))
    bad[3, 5] = True
    assert torch.equal(torch.isnan(stands_for), bad)
    want, _ = quantized(torch.nan_to_num(x.double(), nan=0.0, neginf=0.0), "e4m3", kind)
    assert torch.equal(q.values()[~bad], want[~bad])


def test_quantize_other_stream_and_graph():
    x = Rows(200, 272, torch.bfloat16).set(activations((200, 272), torch.bfloat16, 9))
    q, s = Values(200, 272, "e4m3"), table((3, 200))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        B.gemm_scaled_quantize(0, x, 272, 200, 272, B.GEMM_BF16, 0, q, 272, s, torch.cuda.current_stream())
    for seed in (1, 2):
        x.set(activations((200, 272), torch.bfloat16, seed))
        graph.replay()
        want, scales = quantized(x.view.double(), "e4m3", "rows")
        assert torch.equal(q.values(), want) and torch.equal(s.view, scales.float())


# ---------------------------------------------------------------- norm
EPS = 1e-5


def relative(H):
    """Of rstd: a sum of H squares of 16-bit values in fp32, halved by the root, the mean's and eps's
    roundings, and the root's."""
    return ((H + 3) / 2 + 1) * 2.0 ** -24


def run_norm(rows, H, dtype, residual, out, type="e4m3", ld=0, off=0, seed=0, in_place=False, eps=EPS):
    code, dt = DTYPES[dtype]
    x = Rows(rows, H, dt, H + ld, off).set(activations((rows, H), dt, seed))
    r = Rows(rows, H, dt, H + ld, off).set(activations((rows, H), dt, seed + 1)) if residual else None
    w = Rows(1, H, dt, None, off).set(1 + 0.3 * activations((1, H), dt, seed + 2))
    s64 = x.view.double() if not residual else (x.view.float() + r.view.float()).to(dt).double()
    s = (r if in_place else Rows(rows, H, dt, H + ld, off)) if residual else None
    y = Rows(rows, H, dt, H + ld, off) if out != "q" else None
    q = Values(rows, H, type, H + ld, off) if out != "y" else None
    scales = table((up(H), rows)) if out != "y" else None
    rstd = table((1, rows))
    B.gemm_rms_norm(x, x.ld, r, H + ld, w, eps, rows, H, code, s, H + ld, y, H + ld, q, H + ld, FP8[type][0], scales, rstd)
    for t in (x, r, w, s, y, q, scales, rstd):
        if t is not None:
            t.check_guards()
    if residual:
        assert torch.equal(s.view.double(), s64)
    want_rstd = (s64.square().mean(1) + eps).rsqrt()
    e = relative(H)
    assert bool(((rstd.view[0].double() - want_rstd).abs() <= e * want_rstd).all())
    want = s64 * want_rstd[:, None] * w.view.double()
    e += 2 * 2.0 ** -24  # two products
    if y is not None:
        u, tiny = ROUNDOFF[dt]
        err = (y.view.double() - want).abs()
        assert bool((err <= (e + u * (1 + e)) * want.abs() + tiny).all())
    if q is not None:
        _, _, largest, digits, least = FP8[type]
        m = magnitudes(want, "rows") / largest
        assert bool(((scales.view.double() - m).abs() <= (e + 2.0 ** -24) * 1.01 * m).all())
        # half a step of the value (or of the smallest), of a value within e, a scale within e + 2^-24,
        # and two roundings on the way to the border
        sc = spread(scales.view.double(), rows, H, "rows")
        half = torch.maximum(2.0 ** -(digits + 1) * want.abs(), 2.0 ** (least - digits - 1) * sc)
        err = (q.values() * sc - want).abs()
        assert bool((err <= half * (1 + 4 * e) + 4 * (e + 2.0 ** -23) * want.abs()).all())
    return x, s64, w, rstd


NORM_SIZES = [(1, 1), (1, 128), (1, 4096), (2, 8), (3, 129), (5, 250), (17, 256), (33, 1000), (7, 2056), (300, 264), (20, 4104),
              (3, 8192), (2, 16384), (2, 20011), (1, 32768), (2, 32767), (700, 8200), (800, 3000), (160, 17000)]


@pytest.mark.parametrize("rows,H", NORM_SIZES)
@pytest.mark.parametrize("dtype,residual,out,type", [("bf16", True, "q", "e4m3"), ("f16", False, "y", "e4m3"), ("bf16", True, "both", "e5m2"),
                                                     ("f16", True, "q", "e4m3")])
def test_norm(rows, H, dtype, residual, out, type):
    run_norm(rows, H, dtype, residual, out, type, seed=rows + H)


@pytest.mark.parametrize("ld,off", [(8, 0), (8, 8), (1, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_strides(ld, off, in_place):
    run_norm(40, 520, "bf16", True, "both", ld=ld, off=off, seed=4, in_place=in_place)


def test_norm_rows_of_zeros_and_nan():
    """A row of zeros has rstd 1 / sqrt(eps) and an output of zeros; a NaN stays in its row."""
    H = 512
    x = activations((4, H), torch.bfloat16, 8)
    x[1] = 0
    x[2, 100] = float("nan")
    x = Rows(4, H, torch.bfloat16).set(x)
    w = Rows(1, H, torch.bfloat16).set(torch.ones(1, H, device="cuda"))
    y, q, scales, rstd = Rows(4, H, torch.bfloat16), Values(4, H, "e4m3"), table((4, 4)), table((1, 4))
    B.gemm_rms_norm(x, H, None, 0, w, EPS, 4, H, B.GEMM_BF16, None, 0, y, H, q, H, 0, scales, rstd)
    nan = torch.isnan(y.view).any(1).tolist()
    assert nan == [False, False, True, False] == torch.isnan(q.values()).any(1).tolist()
    assert not y.view[1].any() and not q.values()[1].any() and bool((scales.view[:, 1] == 2.0 ** -100 / 448).all())
    assert abs(float(rstd.view[0, 1]) * EPS ** 0.5 - 1) < 1e-6


def run_grad(rows, H, dtype, dsum, dweight=True, ld=0, off=0, seed=0, alias=None):
    code, dt = DTYPES[dtype]
    make = lambda n: Rows(rows, H, dt, H + ld, off).set(activations((rows, H), dt, seed + n, 0.5))  # noqa: E731
    s, dy, d = make(0), make(1), make(2) if dsum else None
    w = Rows(1, H, dt, None, off).set(1 + 0.3 * activations((1, H), dt, seed + 3))
    rstd = table((1, rows)).set((s.view.double().square().mean(1) + EPS).rsqrt()[None])
    dx = {None: None, "dy": dy, "dsum": d}[alias] or Rows(rows, H, dt, H + ld, off)
    dw = table((1, H)) if dweight else None
    S, DY, W, R = s.view.double(), dy.view.double(), w.view.double(), rstd.view[0].double()[:, None]
    D = d.view.double() if dsum else torch.zeros_like(S)
    ws = torch.full((B.gemm_rms_norm_grad_workspace_size(rows, H) + 16,), 255, dtype=torch.uint8, device="cuda")  # NaN
    B.gemm_rms_norm_grad(dy, dy.ld, s, s.ld, w, rstd, d, H + ld, rows, H, code, dx, dx.ld, dw, ws if dweight else None)
    for t in (s, dy, w, rstd, dx, dw, d):
        if t is not None:
            t.check_guards()
    n = S * R
    p = W * DY * n
    want = R * (W * DY - n * p.mean(1, keepdim=True)) + D
    # each product and sum rounds once, the mean as a sum of H of them
    mean_abs = p.abs().mean(1, keepdim=True)
    e = 2.0 ** -24 * 1.01 * (R * (4 * (W * DY).abs() + n.abs() * mean_abs * (H + 8)) + 2 * want.abs() + D.abs())
    u, tiny = ROUNDOFF[dt]
    err = (dx.view.double() - want).abs()
    assert bool((err <= e + u * (want.abs() + e) + tiny).all()), float((err / (e + u * want.abs() + tiny)).max())
    if dweight:
        want = (DY * n).sum(0)
        e = (rows + 2) * 2.0 ** -24 * 1.01 * (DY * n).abs().sum(0)
        assert bool(((dw.view[0].double() - want).abs() <= e + 2.0 ** -149).all())


@pytest.mark.parametrize("rows,H", NORM_SIZES + [(1000, 512), (2000, 136)])
@pytest.mark.parametrize("dtype,dsum,dweight", [("bf16", True, True), ("f16", False, True), ("bf16", True, False)])
def test_norm_grad(rows, H, dtype, dsum, dweight):
    run_grad(rows, H, dtype, dsum, dweight, seed=rows + H)


@pytest.mark.parametrize("ld,off", [(8, 0), (8, 8), (1, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("alias", [None, "dy", "dsum"])
def test_norm_grad_strides(ld, off, alias):
    run_grad(40, 520, "bf16", True, ld=ld, off=off, seed=4, alias=alias)


def test_norm_grad_repeats_bitwise_and_without_rows():
    H, rows = 1024, 3000
    s, dy = activations((rows, H), torch.bfloat16, 1), activations((rows, H), torch.bfloat16, 2)
    w = activations((1, H), torch.bfloat16, 3)
    rstd = torch.rand(rows, device="cuda") + 0.5
    ws = torch.empty(B.gemm_rms_norm_grad_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(3):
        dx, dw = torch.empty_like(s), torch.empty(H, device="cuda")
        B.gemm_rms_norm_grad(dy, H, s, H, w, rstd, None, 0, rows, H, B.GEMM_BF16, dx, H, dw, ws)
        outs.append((dx, dw))
    assert all(torch.equal(a[0], outs[0][0]) and torch.equal(a[1], outs[0][1]) for a in outs)
    dw.fill_(7)
    B.gemm_rms_norm_grad(None, H, None, H, None, None, None, 0, 0, H, B.GEMM_BF16, None, H, dw, None)
    assert not dw.any()


def test_norm_grad_against_automatic_differentiation():
    """In 64 bits, from the norm's definition, with the residual stream's own gradient."""
    R, H = 37, 200
    x, r, dy, ds = (activations((R, H), torch.float16, n, 0.2) for n in range(4))
    w = (1 + 0.2 * activations((1, H), torch.float16, 5)).half()
    s, y = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(R, device="cuda")
    B.gemm_rms_norm(x, H, r, H, w, EPS, R, H, B.GEMM_F16, s, H, y, H, None, 0, 0, None, rstd)
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.empty(B.gemm_rms_norm_grad_workspace_size(R, H), dtype=torch.uint8, device="cuda")
    B.gemm_rms_norm_grad(dy, H, s, H, w, rstd, ds, H, R, H, B.GEMM_F16, dx, H, dw, ws)
    S, W = s.double().requires_grad_(), w.double().requires_grad_()
    (S * (S.square().mean(1, keepdim=True) + EPS).rsqrt() * W).backward(dy.double())
    want = S.grad + ds.double()
    size = S.grad.abs() + ds.double().abs() + 1
    # the 16-bit rounding, and rstd's error (relative(H), twice: factor and mean) on terms below 4
    assert bool(((dx.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -25 + 8 * relative(H) * 4 * size).all())
    n = s.double() * rstd.double()[:, None]
    e = ((R + 2) * 2.0 ** -24 + relative(H)) * 1.01 * (dy.double() * n).abs().sum(0)
    assert bool(((dw.double() - W.grad[0]).abs() <= e).all())


def test_offsets_past_32_bits():
    """2.3 G elements: the last rows of every form."""
    R, H = 70016, 32768
    x = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
    some = activations((1024, H), torch.bfloat16, 1)
    for at in range(0, R, 1024):
        x[at:at + 1024] = some[:min(1024, R - at)]
    x[-7:] = activations((7, H), torch.bfloat16, 2)
    last = slice(R - 128 - R % 128, R)
    q, s, qc, sc = (torch.empty(R, H, dtype=torch.uint8, device="cuda"), torch.empty(up(H), R, device="cuda"),
                    torch.empty(R, H, dtype=torch.uint8, device="cuda"), torch.empty(up(R), H, device="cuda"))
    B.gemm_scaled_quantize_both(x, H, R, H, B.GEMM_BF16, 0, q, H, s, qc, H, sc)
    part = x[last].double()
    want, scales = quantized(part, "e4m3", "rows")
    assert torch.equal(q[last].view(torch.float8_e4m3fn).double(), want) and torch.equal(s[:, last], scales.float())
    want, scales = quantized(part, "e4m3", "cols")
    assert torch.equal(qc[last].view(torch.float8_e4m3fn).double(), want) and torch.equal(sc[-scales.shape[0]:], scales.float())
    q.zero_()
    B.gemm_scaled_quantize(B.GEMM_QUANTIZE_ROWS, x, H, R, H, B.GEMM_BF16, 0, q, H, s)
    want, _ = quantized(part, "e4m3", "rows")
    assert torch.equal(q[last].view(torch.float8_e4m3fn).double(), want)
    del qc, sc
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    rstd, y = torch.empty(R, device="cuda"), torch.empty_like(x)
    B.gemm_rms_norm(x, H, None, 0, w, EPS, R, H, B.GEMM_BF16, None, 0, y, H, q, H, 0, s, rstd)
    want_rstd = (part.square().mean(1) + EPS).rsqrt()
    assert bool(((rstd[last].double() - want_rstd).abs() <= relative(H) * want_rstd).all())
    want = part * want_rstd[:, None]
    assert bool(((y[last].double() - want).abs() <= (2.0 ** -8 + 2 * relative(H)) * want.abs()).all())
    B.gemm_rms_norm_grad(y, H, x, H, w, rstd, None, 0, R, H, B.GEMM_BF16, y, H, None, None)  # dy is the normed row itself: no gradient
    # y = n + d with |d| <= 2^-8 |n|, so dx = rstd (d + n (1 - mean n^2) - n mean(d n)), where mean n^2 is 1 - eps
    # rstd^2 within twice rstd's error, and the sums round as in run_grad; dx rounds once more
    r = rstd[last].double()[:, None]
    n = part * r
    square = n.square().mean(1, keepdim=True)
    bound = r * n.abs() * (2.0 ** -8 * (1 + square) + EPS * r ** 2 + 2 * relative(H) + (H + 8) * 2.0 ** -24 * square)
    assert bool((y[last].double().abs() <= bound * 1.01 + 2.0 ** -100).all())
