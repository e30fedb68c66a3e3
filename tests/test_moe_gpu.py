"""GPU tests of the mixture-of-experts row operators (sort, dispatch, combine
and their gradients) against 64-bit restatements of their definitions."""
import numpy as np
import pytest
import torch

from persistent_stream_matmul_gb300 import _binding as B
from tests.gpu_util import ensure_built
from tests.moe_util import (DTYPES, Rows, assert_rounded_sum, normal, routing, sorted_slots)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _sort(ids, experts, id_type=torch.int64, pad=0, stream=None):
    """gemm_moe_sort on the device, every output checked for its guards."""
    T, k = ids.shape
    dev = torch.full((max(T, 1), k + pad), 3, dtype=id_type, device="cuda")
    dev[:T, :k] = torch.from_numpy(ids).clamp(torch.iinfo(id_type).min, torch.iinfo(id_type).max).to(id_type)
    outs = [Rows(1, n, torch.int32) for n in (experts + 1, T * k, T * k)]
    ws = torch.randint(0, 256, (max(1, B.gemm_moe_sort_workspace_size(T, k, experts)),), dtype=torch.uint8,
                       device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    B.gemm_moe_sort(dev, B.GEMM_INDEX_I64 if id_type == torch.int64 else B.GEMM_INDEX_I32, k + pad, T, k, experts,
                    *outs, ws, stream)
    torch.cuda.synchronize()
    for o in outs:
        o.check_guards()
    return [o.view[0].cpu().numpy() for o in outs]


SORTS = [(0, 2, 4), (1, 1, 1), (1, 8, 64), (3, 1, 1024), (7, 3, 5), (33, 31, 2), (129, 8, 8), (1000, 2, 8),
         (1023, 1, 3), (1024, 1, 257), (1365, 3, 17), (4096, 1, 64), (4097, 6, 64), (8191, 2, 1000),
         (16385, 4, 1024), (20000, 1, 1), (32768, 8, 256)]


@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,E", SORTS)
def test_sort_equals_stable_sort(T, k, E, id_type):
    for drop, skew, pad in ((0.0, 0.0, 0), (0.2, 1.2, 3)):
        ids = routing(T, k, E, 5 * T + k, drop, skew)
        for got, want in zip(_sort(ids, E, id_type, pad), sorted_slots(ids, E)):
            assert np.array_equal(got, want)


@pytest.mark.parametrize("T,k,E", [(5, 2, 4), (3000, 4, 33), (20001, 2, 128)])
def test_sort_one_expert_none_and_wrapped_values(T, k, E):
    same = np.full((T, k), E - 1, dtype=np.int64)
    # values whose low 32 bits name an expert, which an int64 choice does not
    wrapped = np.full((T, k), 2 ** 32 + 1, dtype=np.int64)
    for ids in (same, np.full((T, k), -1, dtype=np.int64), wrapped):
        for got, want in zip(_sort(ids, E), sorted_slots(ids, E)):
            assert np.array_equal(got, want)


def test_sort_repeats_and_streams():
    ids = routing(12345, 3, 77, 9, 0.1, 0.7)
    first = _sort(ids, 77)
    side = torch.cuda.Stream()
    for got in (_sort(ids, 77), _sort(ids, 77, stream=side)):
        assert all(np.array_equal(a, b) for a, b in zip(first, got))


# ---------------------------------------------------------------- row movements
def _setup(T, k, E, seed, drop):
    ids = routing(T, k, E, seed, drop, 0.5)
    offsets, rows, slots = sorted_slots(ids, E)
    return offsets, rows, slots, torch.from_numpy(rows).cuda(), torch.from_numpy(slots).cuda()


# (tokens, choices, experts, hidden, ld padding, element offset, dropped share):
# one token, odd and tiny rows, rows that start off a 16-byte boundary by ld or
# by offset, a token whose slots are all dropped, more choices than a warp
ROWS = [(1, 1, 1, 8, 0, 0, 0.0), (1, 8, 16, 2048, 0, 0, 0.0), (5, 2, 3, 1, 0, 0, 0.0), (9, 3, 4, 7, 1, 1, 0.3),
        (64, 2, 8, 4096, 0, 0, 0.0), (77, 4, 9, 1000, 8, 0, 0.2), (77, 4, 9, 1000, 4, 0, 0.2),
        (40, 6, 64, 2056, 0, 8, 0.5), (40, 6, 64, 2056, 0, 3, 0.5), (13, 5, 7, 2049, 0, 0, 0.1),
        (3, 40, 50, 264, 0, 0, 0.3), (257, 8, 32, 768, 0, 0, 1.0), (1025, 2, 4, 520, 0, 0, 0.05),
        (6, 3, 4, 16392, 0, 0, 0.2), (2, 2, 2, 40000, 0, 0, 0.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,E,H,pad,off,drop", ROWS)
def test_dispatch_and_gradient(T, k, E, H, pad, off, drop, dtype):
    code, dt = DTYPES[dtype]
    _, rows, slots, drows, dslots = _setup(T, k, E, T + H, drop)
    x = Rows(T, H, dt, H + pad, off).set(normal((T, H), dt, 1))
    xs = Rows(T * k, H, dt, H + pad, off)
    B.gemm_moe_dispatch(x, x.ld, drows, dslots, T, k, H, code, xs, xs.ld)
    want = torch.zeros((T * k, H), dtype=dt, device="cuda")
    used = torch.from_numpy(np.flatnonzero(slots >= 0)).cuda()
    want[used] = x.view[torch.from_numpy(slots[slots >= 0] // k).long().cuda()]
    assert torch.equal(xs.view, want)
    xs.check_guards()

    dxs = Rows(T * k, H, dt, H + pad, off).set(normal((T * k, H), dt, 2))
    dxs.view[int((slots >= 0).sum()):] = float("nan")  # unused rows are not read
    dx = Rows(T, H, dt, H + pad, off)
    B.gemm_moe_dispatch_grad(dxs, dxs.ld, drows, T, k, H, code, dx, dx.ld)
    exact = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    absolute = torch.zeros_like(exact)
    for s, r in enumerate(rows.tolist()):
        if r >= 0:
            exact[s // k] += dxs.view[r].double()
            absolute[s // k] += dxs.view[r].double().abs()
    assert_rounded_sum(dx.view, exact, absolute, k)
    dx.check_guards()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,E,H,pad,off,drop", ROWS)
def test_combine_and_gradient(T, k, E, H, pad, off, drop, dtype):
    code, dt = DTYPES[dtype]
    _, rows, slots, drows, dslots = _setup(T, k, E, T + H + 1, drop)
    used = int((slots >= 0).sum())
    ys = Rows(T * k, H, dt, H + pad, off).set(normal((T * k, H), dt, 3))
    ys.view[used:] = float("nan")
    w = torch.rand(T * k, generator=torch.Generator().manual_seed(4)).cuda()
    w[drows < 0] = float("nan")  # a dropped slot's weight is not read
    y = Rows(T, H, dt, H + pad, off)
    B.gemm_moe_combine(ys, ys.ld, drows, w, T, k, H, code, y, y.ld)
    exact = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    absolute = torch.zeros_like(exact)
    for s, r in enumerate(rows.tolist()):
        if r >= 0:
            term = w[s].double() * ys.view[r].double()
            exact[s // k] += term
            absolute[s // k] += term.abs()
    assert_rounded_sum(y.view, exact, absolute, k)
    y.check_guards()

    dy = Rows(T, H, dt, H + pad, off).set(normal((T, H), dt, 5))
    dys = Rows(T * k, H, dt, H + pad, off)
    dw = Rows(1, T * k, torch.float32)
    B.gemm_moe_combine_grad(dy, dy.ld, ys, ys.ld, drows, dslots, w, T, k, H, code, dys, dys.ld, dw)
    edys = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
    edw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    adw = torch.zeros_like(edw)
    for s, r in enumerate(rows.tolist()):
        if r >= 0:
            edys[r] = w[s].double() * dy.view[s // k].double()
            terms = dy.view[s // k].double() * ys.view[r].double()
            edw[s], adw[s] = terms.sum(), terms.abs().sum()
    assert_rounded_sum(dys.view, edys, edys.abs(), 1)
    assert bool((dys.view[used:] == 0).all()) and not bool(torch.signbit(dys.view[used:]).any())
    # an fp32 sum of H exact products in any order
    assert bool(((dw.view[0].double() - edw).abs() <= (H + 1) * 2.0 ** -24 * 1.01 * adw).all())
    dys.check_guards()
    dw.check_guards()


def test_infinite_and_nan_rows_stay_in_their_tokens():
    T, k, E, H = 12, 2, 4, 72
    _, rows, slots, drows, _ = _setup(T, k, E, 3, 0.0)
    ys = normal((T * k, H), torch.bfloat16, 6)
    ys[int(rows[0])] = float("inf")
    ys[int(rows[2 * k])] = float("nan")
    w = torch.full((T * k,), 0.5, device="cuda")
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    B.gemm_moe_combine(ys, H, drows, w, T, k, H, B.GEMM_BF16, y, H)
    assert bool(torch.isinf(y[0]).all()) and bool(torch.isnan(y[2]).all())
    assert bool(torch.isfinite(y[[1, *range(3, T)]]).all())


def test_rows_out_of_range_count_as_dropped():
    T, k, H = 4, 2, 16
    rows = torch.tensor([0, 8, 1, 2 ** 31 - 1, -5, 2, 3, -2 ** 31], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 2, 5, 6, -1, -1, -1, -1], dtype=torch.int32, device="cuda")
    x = normal((T, H), torch.float16, 7)
    xs = Rows(T * k, H, torch.float16)
    B.gemm_moe_dispatch(x, H, rows, slots, T, k, H, B.GEMM_F16, xs, H)
    want = torch.zeros((T * k, H), dtype=torch.float16, device="cuda")
    want[0], want[1], want[2], want[3] = x[0], x[1], x[2], x[3]
    assert torch.equal(xs.view, want)
    xs.check_guards()
    dx = torch.empty((T, H), dtype=torch.float16, device="cuda")
    B.gemm_moe_dispatch_grad(xs, H, rows, T, k, H, B.GEMM_F16, dx, H)
    assert torch.equal(dx, x)


def test_large_offsets_pass_32_bits():
    """Row r at r * ld elements lies past 2^32 elements: the last rows of a
    wide-strided matrix, moved both ways."""
    T, k, H, ld = 5, 1, 24, 2 ** 30 + 8
    buf = torch.zeros((T - 1) * ld + H, dtype=torch.bfloat16, device="cuda")  # 8.6 GB
    wide = torch.as_strided(buf, (T, H), (ld, 1))
    rows = torch.tensor([4, 3, 2, 1, 0], dtype=torch.int32, device="cuda")
    x = normal((T, H), torch.bfloat16, 8)
    B.gemm_moe_dispatch(x, H, rows, rows, T, k, H, B.GEMM_BF16, buf, ld)
    assert torch.equal(wide, x.flip(0))
    back = torch.empty_like(x)
    B.gemm_moe_dispatch_grad(buf, ld, rows, T, k, H, B.GEMM_BF16, back, H)
    assert torch.equal(back, x)


def test_operators_follow_their_stream():
    """On a side stream behind a long wait, the chain reads what the stream
    wrote before it, and a captured graph replays it on new inputs."""
    T, k, E, H = 300, 2, 8, 512
    ids = torch.from_numpy(routing(T, k, E, 11, 0.1)).cuda()
    x = normal((T, H), torch.bfloat16, 9)
    w = torch.rand(T * k, device="cuda")
    offsets, rows, slots = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
    ws = torch.empty(max(1, B.gemm_moe_sort_workspace_size(T, k, E)), dtype=torch.uint8, device="cuda")
    xin, xs = torch.zeros_like(x), torch.empty((T * k, H), dtype=x.dtype, device="cuda")
    y = torch.empty_like(x)

    def chain(stream):
        B.gemm_moe_sort(ids, B.GEMM_INDEX_I64, k, T, k, E, offsets, rows, slots, ws, stream)
        B.gemm_moe_dispatch(xin, H, rows, slots, T, k, H, B.GEMM_BF16, xs, H, stream)
        B.gemm_moe_combine(xs, H, rows, w, T, k, H, B.GEMM_BF16, y, H, stream)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        xin.copy_(x)
        chain(side)
        got = y.clone()
    side.synchronize()
    wsum = torch.where(rows >= 0, w, 0.0).reshape(T, k)
    exact = wsum.double().sum(1)[:, None] * x.double()
    assert_rounded_sum(got, exact, exact.abs(), k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(torch.cuda.current_stream())
    for seed in (21, 22):
        xin.copy_(normal((T, H), torch.bfloat16, seed))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        exact = wsum.double().sum(1)[:, None] * xin.double()
        assert_rounded_sum(y, exact, exact.abs(), k)


def test_combine_gradient_against_differences():
    """L = <dy, combine(ys, w)> is linear in ys and in w, so its difference
    quotient equals the gradient up to the rounding of the two outputs: each
    y element is within (u + 2^-20) of its magnitude, so L within that of
    sum |dy| |y|, whatever the step."""
    T, k, E, H = 10, 3, 5, 200
    _, rows, slots, drows, dslots = _setup(T, k, E, 5, 0.1)
    dt = torch.float16
    ys, dy = normal((T * k, H), dt, 12), normal((T, H), dt, 13)
    w = torch.rand(T * k, device="cuda")
    dys, dw = torch.empty_like(ys), torch.empty_like(w)
    B.gemm_moe_combine_grad(dy, H, ys, H, drows, dslots, w, T, k, H, B.GEMM_F16, dys, H, dw)

    def loss(ys, w):
        y = torch.empty((T, H), dtype=dt, device="cuda")
        B.gemm_moe_combine(ys, H, drows, w, T, k, H, B.GEMM_F16, y, H)
        per = dy.double() * y.double()
        return per.sum().item(), per.abs().sum().item()

    step = 4.0
    for s in range(0, T * k, 4):
        wp, wm = w.clone(), w.clone()
        wp[s] += step
        wm[s] -= step
        (lp, mp), (lm, mm) = loss(ys, wp), loss(ys, wm)
        h = (wp[s] - wm[s]).item()
        assert abs((lp - lm) / h - dw[s].item()) <= (2.0 ** -11 + 2.0 ** -20) * (mp + mm) / h + 1e-4
    for r in range(0, T * k, 5):
        yp, ym = ys.clone(), ys.clone()
        yp[r, 17] += 8
        ym[r, 17] -= 8
        h = (yp[r, 17].double() - ym[r, 17].double()).item()
        (lp, mp), (lm, mm) = loss(yp, w), loss(ym, w)
        assert abs((lp - lm) / h - dys[r, 17].item()) <= (2.0 ** -11 + 2.0 ** -20) * (mp + mm) / h + 4e-3
