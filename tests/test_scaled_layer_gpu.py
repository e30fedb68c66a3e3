"""The 8-bit feed-forward layer: every step of its chain against the step's 64-bit
value for the operands that the layer itself made, the whole chain bit for bit on
inputs that 8 bits hold, and its refusals."""
import pytest
import torch

from persistent_stream_matmul_gb300 import _binding as B
from persistent_stream_matmul_gb300.scaled_layer import ScaledFeedForward
from tests.gpu_util import ensure_built
from tests.scaled_util import assert_product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _signs(shape, seed, share):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.rand(shape, generator=g, device="cuda")
    return ((v < share / 2).int() - (v > 1 - share / 2).int()).half()


@pytest.mark.parametrize("T,H,F", [(1, 64, 128), (5, 128, 272), (40, 256, 144), (300, 128, 400), (700, 272, 512)])
@pytest.mark.parametrize("grad_type", [B.GEMM_E4M3, B.GEMM_E5M2])
def test_layer_equals_its_formulas(T, H, F, grad_type):
    """Rows of s are +-1, so rstd = 1 for eps = 0 and the normed row is s.  A group of values in -m, 0, m
    stands for itself in 8 bits.  up and down have one element of +-1 a row, so the activations and y
    are -1, 0 or 1: forward is exact."""
    x = torch.where(_signs((T, H), 1, 1.0) >= 0, 1.0, -1.0).half()
    residual = torch.zeros_like(x)
    norm = torch.ones(H, device="cuda").half()
    up, down = torch.zeros(F, H, device="cuda").half(), torch.zeros(H, F, device="cuda").half()
    g = torch.Generator(device="cuda").manual_seed(3)
    up[torch.arange(F), torch.randint(H, (F,), generator=g, device="cuda")] = torch.where(torch.rand(F, generator=g, device="cuda") < 0.5, 1.0, -1.0).half()
    down[torch.arange(H), torch.randint(F, (H,), generator=g, device="cuda")] = torch.where(torch.rand(H, generator=g, device="cuda") < 0.5, 1.0, -1.0).half()
    layer = ScaledFeedForward(T, norm, up, down, eps=0.0, grad_type=grad_type)
    y, s = layer.forward(x, residual)
    dy = _signs((T, H), 5, 0.3)
    ds = _signs((T, H), 6, 0.3)
    a = layer.saved[3]
    X, U, D = x.double(), up.double(), down.double()
    A = torch.relu(X @ U.t())
    assert torch.equal(s, x) and torch.equal(a.double(), A) and torch.equal(y.double(), A @ D.t())
    dx, dnorm, dup, ddown = layer.backward(dy, ds)
    layer.check()
    # the one sum of many products: the scale 1 / 448 is rounded (2^-24), so a product is 1 within
    # 2^-23, one of the three roundings that the bound of a product leaves for its scales
    assert_product(ddown, dy.double().t() @ A, dy.double().abs().t() @ A, T)
    dA = (dy.double() @ D) * (A > 0)
    # sums of several signs need not survive 8 bits: what follows is held to the format's half step
    step = 2.0 ** -4 if grad_type == B.GEMM_E4M3 else 2.0 ** -3
    bound = step * (dA.abs().t() @ X.abs()) * 1.01 + 2.0 ** -10 * (dA.t() @ X).abs() + 1e-3
    assert bool(((dup.double() - dA.t() @ X).abs() <= bound).all())
    dn = dA @ U
    e = step * (dA.abs() @ U.abs()) * 1.01 + 2.0 ** -10 * dn.abs()
    want = dn - X * (dn * X).mean(1, keepdim=True) + ds.double()
    assert bool(((dx.double() - want).abs() <= e + e.mean(1, keepdim=True) + 2.0 ** -10 * want.abs() + 1e-3).all())
    assert bool(((dnorm.double() - (dn * X).sum(0)).abs() <= e.sum(0) + 1e-3 * (1 + T / 64)).all())
    layer.close()


@pytest.mark.parametrize("T,H,F", [(1, 512, 1024), (130, 512, 768), (600, 1024, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer_is_near_the_16_bit_chain(T, H, F, dtype):
    """Against 64 bits and automatic differentiation, as a whole.  In norm, normal values in e4m3 are
    0.026 off and in e5m2 0.051 (a value in [2^e, 2^(e+1)) is off by up to half a step, evenly), and errors of
    independent signs add in squares.  y passes four e4m3 operands: 0.026 * 2 = 0.052.  An activation is
    0.026 * sqrt(2) = 0.037 of its size off before ReLU, so its sign turns with probability
    arctan(0.037) / pi = 0.0117; where it does, the gradient is masked the other way, which is
    0.0117 / 0.5 of its energy. With two operands in e5m2 and two in e4m3 that is sqrt(0.0234 + 2 * 0.051^2 +
    2 * 0.026^2) = 0.173. A third is left for the chance of the draw."""
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *shape, scale=1.0: (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)  # noqa: E731
    x, r, dy, ds = n(T, H), n(T, H), n(T, H), n(T, H)
    norm, up, down = (1 + 0.1 * n(H).float()).to(dtype), n(F, H, scale=H ** -0.5), n(H, F, scale=F ** -0.5)
    layer = ScaledFeedForward(T, norm, up, down)
    y, s = layer.forward(x, r)
    dx, dnorm, dup, ddown = layer.backward(dy, ds)
    layer.check()
    S, W, U, D = (v.double().requires_grad_() for v in (s, norm, up, down))
    Y = torch.relu((S * (S.square().mean(1, keepdim=True) + 1e-5).rsqrt() * W) @ U.t()) @ D.t()
    Y.backward(dy.double())
    far = lambda got, want: float((got.double() - want).norm() / want.norm())  # noqa: E731
    assert far(y, Y.detach()) < 0.052 * 4 / 3
    for got, want in ((dx.double() - ds.double(), S.grad), (dnorm, W.grad), (dup, U.grad), (ddown, D.grad)):
        assert far(got, want) < 0.173 * 4 / 3
    y2, s2 = layer.forward(x, r, train=False)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    with pytest.raises(RuntimeError):
        layer.backward(dy)
    layer.close()


def test_layer_captured_on_another_stream():
    T, H, F = 200, 256, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    layer = ScaledFeedForward(T, n(H), n(F, H), n(H, F))
    x, r, dy = n(T, H), n(T, H), n(T, H)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        y, s = layer.forward(x, r)
        grads = layer.backward(dy, s)
    for _ in range(3):
        for t in (x, r, dy):
            t.copy_(n(T, H))
        graph.replay()
        torch.cuda.synchronize()
        want_y, want_s = layer.forward(x, r)
        want = layer.backward(dy, want_s)
        assert torch.equal(y, want_y) and torch.equal(s, want_s) and all(torch.equal(a, b) for a, b in zip(grads, want))
    layer.check()


def test_layer_refuses_other_operands():
    T, H, F = 16, 64, 128
    w = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    for bad in ((w(H + 1), w(F, H), w(H, F)), (w(H), w(F, H), w(F, H)), (w(H), w(F, H), w(H, F, dtype=torch.float16)),
                (w(H), w(F, H).float(), w(H, F)), (w(H), w(F, H), w(F, H).t()), (w(H), w(F, H).cpu(), w(H, F))):
        with pytest.raises(ValueError):
            ScaledFeedForward(T, *bad)
    with pytest.raises(ValueError):
        ScaledFeedForward(T, w(H), w(F, H), w(H, F), grad_type=7)
    layer = ScaledFeedForward(T, w(H), w(F, H), w(H, F))
    with pytest.raises(RuntimeError):
        layer.backward(w(T, H))
    for bad in ((w(T, H + 1), w(T, H)), (w(T, H), w(T + 1, H)), (w(T, H).half(), w(T, H)), (w(H, T).t(), w(T, H)), (w(T, H).cpu(), w(T, H))):
        with pytest.raises(ValueError):
            layer.forward(*bad)
    layer.forward(w(T, H), w(T, 2 * H)[:, :H])  # any row stride
    with pytest.raises(ValueError):
        layer.backward(w(T, H + 1))
    with pytest.raises(ValueError):
        layer.backward(w(T, H), w(T, H).half())
