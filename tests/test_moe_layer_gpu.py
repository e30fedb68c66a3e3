"""The mixture-of-experts layer, all its operators in one chain, against
automatic differentiation in 64 bits.

Inputs are small whole numbers and weights powers of two, so that every value
of the chain is exact in fp16 and in its fp32 sums: the layer must equal the
64-bit chain without any tolerance."""
import pytest
import torch

from persistent_stream_matmul_gb300.moe_layer import MoELayer
from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _ints(shape, lo, hi, seed, share=1.0):
    """Whole numbers in [lo, hi], a share of them not zero."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(lo, hi + 1, shape, generator=g, device="cuda")
    return (v * (torch.rand(shape, generator=g, device="cuda") < share)).half()


@pytest.mark.parametrize("T,k,E,H,F,drop", [(1, 2, 8, 64, 72, 0.0), (300, 2, 8, 136, 64, 0.2), (2000, 4, 16, 64, 128, 0.0),
                                           (37, 3, 40, 72, 264, 0.5)])
def test_layer_equals_autograd(T, k, E, H, F, drop):
    x, dy = _ints((T, H), -1, 1, 1, 0.5), _ints((T, H), -1, 1, 2, 0.1)
    up, down = _ints((E, F, H), -1, 1, 3, 0.1), _ints((E, H, F), -1, 1, 4, 0.1)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < drop, -1, ids)
    w = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.5, 0.5, 1.0)
    layer = MoELayer(T, k, _ints((E, H), -1, 1, 6), up, down)
    y = layer.forward(x, ids, w)
    dx, dw, dup, ddown = layer.backward(dy)
    layer.check()

    X, U, D, W = (v.double().requires_grad_() for v in (x, up, down, w))
    Y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        Y = Y.index_add(0, t, (torch.relu(X[t] @ U[e].t()) @ D[e].t()) * W[t, j][:, None])
    Y.backward(dy.double())
    for name, got, want in (("y", y, Y), ("dx", dx, X.grad), ("dup", dup, U.grad), ("ddown", ddown, D.grad),
                            ("dw", dw, W.grad)):
        want = want.detach()
        if got.dtype == torch.float16:  # the chain's values are exact in fp16, so the test is too
            assert bool((want.half().double() == want).all()), name
        assert torch.equal(got.double(), want), name
    layer.close()


def test_route_orders_by_logits():
    layer = MoELayer(5, 2, _ints((8, 64), -1, 1, 1), _ints((8, 64, 64), -1, 1, 2), _ints((8, 64, 64), -1, 1, 3))
    x = _ints((5, 64), -1, 1, 4)
    ids, w = layer.route(x)
    logits = x.double() @ layer.router.double().t()
    top = logits.topk(2, dim=1).values
    assert torch.equal(logits.gather(1, ids), top)
    assert torch.allclose(w.double(), torch.softmax(top, dim=1), rtol=1e-6)
    layer.close()


def test_layer_in_a_graph_with_changing_routes():
    """The whole step is captured once; other choices replay it without a
    group size ever reaching the host."""
    T, k, E, H, F = 64, 2, 8, 64, 64
    up, down = _ints((E, F, H), -1, 1, 3, 0.2), _ints((E, H, F), -1, 1, 4, 0.2)
    layer = MoELayer(T, k, _ints((E, H), -1, 1, 6), up, down)
    x, dy, w = _ints((T, H), -1, 1, 1), _ints((T, H), -1, 1, 2), torch.ones(T, k, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int64, device="cuda")
    layer.backward(layer.forward(x, ids, w))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(x, ids, w)
        grads = layer.backward(dy)
    for seed in (7, 8, 9):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids.copy_(torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices)
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (y, *grads)]
        want = [layer.forward(x, ids, w)]
        want += layer.backward(dy)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    layer.close()
