"""The mixture-of-experts layer's operands: strided ones give the same results,
and those that the operators would read wrongly are refused before any launch."""
import pytest
import torch

from persistent_stream_matmul_gb300.moe_layer import MoELayer
from tests.gpu_util import ensure_built
from tests.moe_util import normal

pytestmark = pytest.mark.gpu

T, K, E, H, F = 40, 3, 8, 72, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.fixture
def layer():
    dt = torch.float16
    made = MoELayer(T, K, normal((E, H), dt, 1), normal((E, F, H), dt, 2, 0.1), normal((E, H, F), dt, 3, 0.1))
    yield made
    made.close()


def _operands():
    x, dy = normal((T, H), torch.float16, 4), normal((T, H), torch.float16, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1).indices
    return x, ids, torch.rand(T, K, generator=g, device="cuda"), dy


def test_strided_and_narrow_operands_give_the_same(layer):
    x, ids, w, dy = _operands()
    routed = layer.route(x)
    want = [layer.forward(x, ids, w), *layer.backward(dy)]
    wide = torch.full((T, H + 5), 7, dtype=x.dtype, device="cuda")
    wide[:, 3:3 + H] = x
    wide_dy = torch.full((2 * T, H), 7, dtype=x.dtype, device="cuda")
    wide_dy[::2] = dy
    wide_ids = torch.zeros((T, E), dtype=torch.int64, device="cuda")
    wide_ids[:, 2:2 + K] = ids
    for i in (wide_ids[:, 2:2 + K], ids.int(), wide_ids.int()[:, 2:2 + K]):
        got = [layer.forward(wide[:, 3:3 + H], i, w), *layer.backward(wide_dy[::2])]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(layer.route(wide[:, 3:3 + H]), routed))


def test_one_token_of_any_stride():
    dt = torch.bfloat16
    one = MoELayer(1, K, normal((E, H), dt, 1), normal((E, F, H), dt, 2, 0.1), normal((E, H, F), dt, 3, 0.1))
    x, w = normal((1, H), dt, 4), torch.rand(1, K, device="cuda")
    ids = torch.arange(K, device="cuda")[None]
    strange = x.as_strided((1, H), (1, 1))
    assert torch.equal(one.forward(x, ids, w), one.forward(strange, ids.expand(1, K), w))
    one.close()


def test_operands_that_do_not_fit_are_refused(layer):
    x, ids, w, dy = _operands()
    with pytest.raises(RuntimeError):
        layer.backward(dy)
    good = (x, ids, w)
    bad = [(0, x.float()), (0, x.bfloat16()), (0, x[:-1]), (0, x[:, :-8]), (0, x.cpu()), (0, x.t().contiguous().t()),
           (0, x[:1].expand(T, H)), (0, x[None]), (0, None), (1, ids.short()), (1, ids[:-1]), (1, ids[:, :2]), (1, ids.cpu()),
           (1, ids.float()), (1, ids.t().contiguous().t()), (2, w.half()), (2, w.double()), (2, w.reshape(-1)),
           (2, torch.rand(T, 2 * K, device="cuda")[:, ::2]), (2, w.cpu()), (2, w[:-1])]
    for i, value in bad:
        args = list(good)
        args[i] = value
        with pytest.raises(ValueError):
            layer.forward(*args)
    for value in (x.float(), x[:-1], x.cpu()):
        with pytest.raises(ValueError):
            layer.route(value)
    layer.forward(*good)
    for value in (dy.float(), dy[1:], dy.cpu(), dy[:, :-1], dy.t().contiguous().t()):
        with pytest.raises(ValueError):
            layer.backward(value)
    layer.backward(dy)
    layer.check()


def test_weights_that_do_not_fit_are_refused():
    dt = torch.float16
    good = [normal((E, H), dt, 1), normal((E, F, H), dt, 2), normal((E, H, F), dt, 3)]
    for i, value in ((0, good[0].bfloat16()), (0, good[0][:, :-8]), (0, good[0].cpu()), (1, good[1].float()), (1, good[1][0]),
                     (1, good[1].cpu()), (2, good[2].bfloat16()), (2, good[2].transpose(1, 2)), (2, good[2][:-1]),
                     (1, good[1].transpose(0, 1).contiguous().transpose(0, 1)), (1, None)):
        weights = list(good)
        weights[i] = value
        with pytest.raises(ValueError):
            MoELayer(T, K, *weights)
