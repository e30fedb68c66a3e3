"""GPU tests of the grouped products against 64-bit products of the groups."""
import numpy as np
import pytest
import torch

from persistent_stream_matmul_gb300 import _binding as B
from tests.gpu_util import ensure_built
from tests.moe_util import DTYPES, Rows, assert_rounded_sum, normal

pytestmark = pytest.mark.gpu

COL, ROW = B.GEMM_COL_MAJOR, B.GEMM_ROW_MAJOR


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _sizes(counts, unused=0):
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    return offsets, int(np.sum(counts)) + unused


def _run(kind, counts, unused, N, K, dtype, layout, A, Bm, offsets=None, stream=None, ctas=None):
    """One run with guards around C; returns C in its natural shape."""
    code, dt = DTYPES[dtype]
    E = len(counts)
    offs, R = _sizes(counts, unused)
    offs = offsets if offsets is not None else offs
    plan = B.GroupedPlan(kind, E, R, N, K, code, layout, ctas=ctas)
    C = Rows(1, (R if kind == B.GEMM_GROUPED_ROWS else E * K) * N, dt, offset=64)
    ws = torch.randint(0, 256, (max(1, plan.workspace_size),), dtype=torch.uint8, device="cuda")
    plan.run(A, Bm, C, offs, ws, stream)
    assert plan.last_status(stream) == B.GEMM_OK
    C.check_guards()
    plan.close()
    flat = C.view[0]
    if kind == B.GEMM_GROUPED_ROWS:
        return flat.reshape(R, N)
    return flat.reshape(E, N, K) if layout == COL else flat.reshape(E, K, N)


def _reference(kind, counts, R, N, K, layout, A, Bm):
    E = len(counts)
    rows = kind == B.GEMM_GROUPED_ROWS
    shape = (R, N) if rows else ((E, N, K) if layout == COL else (E, K, N))
    exact = torch.zeros(shape, dtype=torch.float64, device="cuda")
    absolute = torch.zeros_like(exact)
    at = 0
    for e, n in enumerate(counts):
        a, at = A[at:at + n].double(), at + n
        if rows:
            b = Bm[e].double().t() if layout == COL else Bm[e].double()
            exact[at - n:at], absolute[at - n:at] = a @ b, a.abs() @ b.abs()
        else:
            d = Bm[at - n:at].double()
            c, m = a.t() @ d, a.abs().t() @ d.abs()
            exact[e], absolute[e] = (c.t(), m.t()) if layout == COL else (c, m)
    return exact, absolute


def _operands(kind, counts, R, N, K, dtype, layout, seed, integers=False):
    _, dt = DTYPES[dtype]
    E = len(counts)
    shape = ((E, N, K) if layout == COL else (E, K, N)) if kind == B.GEMM_GROUPED_ROWS else (R, N)
    if integers:
        g = torch.Generator(device="cuda").manual_seed(seed)
        A = torch.randint(-2, 3, (R, K), generator=g, device="cuda").to(dt)
        Bm = torch.randint(-2, 3, shape, generator=g, device="cuda").to(dt)
    else:
        A, Bm = normal((R, K), dt, seed), normal(shape, dt, seed + 1, 0.25)
    A[int(np.sum(counts)):] = float("nan")  # unused rows are not read into anything
    if kind == B.GEMM_GROUPED_INNER:
        Bm[int(np.sum(counts)):] = float("nan")
    return A, Bm


# (group sizes, unused rows, N, K): one row; odd sizes around every tile and
# 16-row step; empty groups at both ends and in between; one group; skew; sums
# that split; sizes smaller than a tile in every direction
SHAPES = [
    ([1], 0, 8, 8), ([0, 1, 0], 2, 64, 128), ([1] * 8, 0, 1536, 2048), ([3, 0, 5, 1], 0, 264, 520),
    ([15, 16, 17, 0, 31, 33], 7, 136, 200), ([63, 64, 65, 1], 0, 256, 64), ([127, 129, 0, 255, 257], 3, 384, 320),
    ([300], 0, 520, 1000), ([0, 0, 0], 5, 128, 72), ([511, 0, 1, 513, 40], 0, 1000, 136),
    ([2] * 40, 0, 328, 4096), ([1000, 1, 1, 1], 20, 248, 2304), ([24] * 8, 0, 2048, 1024), ([700, 900], 0, 776, 776),
    ([5, 2000, 3], 0, 256, 512),
]


@pytest.mark.parametrize("layout", [COL, ROW])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", [B.GEMM_GROUPED_ROWS, B.GEMM_GROUPED_INNER])
@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("counts,unused,N,K", SHAPES)
def test_products_of_groups(counts, unused, N, K, ctas, kind, dtype, layout):
    R = int(np.sum(counts)) + unused
    A, Bm = _operands(kind, counts, R, N, K, dtype, layout, 7)
    exact, absolute = _reference(kind, counts, R, N, K, layout, A, Bm)
    got = _run(kind, counts, unused, N, K, dtype, layout, A, Bm, ctas=ctas)
    assert_rounded_sum(got, exact, absolute, K if kind == B.GEMM_GROUPED_ROWS else max(counts))
    again = _run(kind, counts, unused, N, K, dtype, layout, A, Bm, ctas=ctas)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    # whole numbers: every partial sum is exact, so only the last rounding remains
    A, Bm = _operands(kind, counts, R, N, K, dtype, layout, 17, integers=True)
    exact, absolute = _reference(kind, counts, R, N, K, layout, A, Bm)
    got = _run(kind, counts, unused, N, K, dtype, layout, A, Bm, ctas=ctas)
    assert torch.equal(got, exact.to(got.dtype))


# few tiles over a long sum, so that every tile is split: (kind, sizes, unused, N, K)
SPLITS = [
    (0, [1], 0, 64, 8192), (0, [3, 0, 40], 2, 136, 6000), (0, [200], 0, 512, 16384), (0, [0, 300, 0], 0, 264, 4104),
    (0, [16, 1, 16], 0, 8, 20000), (0, [257], 1, 256, 4096), (1, [5000], 3, 264, 136), (1, [4000, 0, 700, 1], 0, 128, 256),
    (1, [16385], 0, 8, 8), (1, [0, 3000, 0], 0, 520, 72), (1, [9999, 5, 2501], 10, 64, 512),
]


@pytest.mark.parametrize("layout", [COL, ROW])
@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("kind,counts,unused,N,K", SPLITS)
def test_split_tiles(kind, counts, unused, N, K, ctas, layout):
    """Partials of several units joined by whoever comes last: within the bound,
    the same bits on every run, whatever the workspace held."""
    R = sum(counts) + unused
    offsets = np.concatenate([[0], np.cumsum(counts)])
    with B.GroupedPlan(kind, len(counts), R, N, K, B.GEMM_BF16, layout, ctas=ctas) as p:
        work = [w for u in range(p.info("units")) for w in p.units(offsets, u)]
        assert any(k1 - k0 < kb for *_, k0, k1, kb in work)  # the case splits
    A, Bm = _operands(kind, counts, R, N, K, "bf16", layout, 23)
    exact, absolute = _reference(kind, counts, R, N, K, layout, A, Bm)
    first = None
    for _ in range(4):
        got = _run(kind, counts, unused, N, K, "bf16", layout, A, Bm, ctas=ctas)
        assert_rounded_sum(got, exact, absolute, K if kind == 0 else max(counts))
        first = got if first is None else first
        assert torch.equal(got.view(torch.int16), first.view(torch.int16))
    A, Bm = _operands(kind, counts, R, N, K, "f16", layout, 24, integers=True)
    exact, _ = _reference(kind, counts, R, N, K, layout, A, Bm)
    assert torch.equal(_run(kind, counts, unused, N, K, "f16", layout, A, Bm, ctas=ctas), exact.half())


@pytest.mark.parametrize("ctas,counts,N,K", [(1, [128 * 100, 128 * 55], 128, 2048), (2, [256 * 60, 0, 256 * 18], 256, 4096),
                                             (1, [20, 19900, 7], 64, 4104), (2, [19968, 300], 200, 3080)])
def test_a_remainder_of_tiles_is_split(ctas, counts, N, K):
    """Tiles that are left over a whole round of the units run in shares before
    the whole ones."""
    R = sum(counts)
    with B.GroupedPlan(0, len(counts), R, N, K, B.GEMM_F16, COL, ctas=ctas) as p:
        work = [p.units(np.concatenate([[0], np.cumsum(counts)]), u) for u in range(p.info("units"))]
        assert any(w[0][7] - w[0][6] < w[0][8] for w in work) and all(w[-1][8] == w[-1][7] for w in work)
    A, Bm = _operands(0, counts, R, N, K, "f16", COL, 31)
    exact, absolute = _reference(0, counts, R, N, K, COL, A, Bm)
    got = _run(0, counts, 0, N, K, "f16", COL, A, Bm, ctas=ctas)
    assert_rounded_sum(got, exact, absolute, K)
    assert torch.equal(got.view(torch.int16), _run(0, counts, 0, N, K, "f16", COL, A, Bm, ctas=ctas).view(torch.int16))


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("kind", [B.GEMM_GROUPED_ROWS, B.GEMM_GROUPED_INNER])
def test_split_tiles_replay_and_share_a_workspace(kind, ctas):
    """A captured launch keeps its run number: replays, other plans' runs in the
    same workspace between them, and sizes that change which tiles split all
    give the bits of a fresh run."""
    E, R, N, K = 3, 9000, 72, 8192 if kind == B.GEMM_GROUPED_ROWS else 136
    code, dt = DTYPES["bf16"]
    sizes = ([2, 0, 5], [700, 8300, 0], [0, 0, 0], [9000, 0, 0], [1, 1, 1])
    A = normal((R, K), dt, 1)
    Bm = normal((E, N, K) if kind == B.GEMM_GROUPED_ROWS else (R, N), dt, 2, 0.25)
    plans = [B.GroupedPlan(kind, E, R, N, K, code, COL, ctas=ctas) for _ in range(2)]
    ws = torch.randint(0, 256, (plans[0].workspace_size,), dtype=torch.uint8, device="cuda")
    C = torch.empty((R, N) if kind == B.GEMM_GROUPED_ROWS else (E, N, K), dtype=dt, device="cuda")
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plans[0].run(A, Bm, C, offs, ws, torch.cuda.current_stream())
    for counts in sizes:
        fresh, _ = _sizes(counts)
        offs.copy_(fresh)
        want = torch.empty_like(C)
        plans[1].run(A, Bm, want, offs, torch.zeros_like(ws), torch.cuda.current_stream())
        for _ in range(3):
            C.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(C.view(torch.int16), want.view(torch.int16))
            C.fill_(7)
            plans[1].run(A, Bm, C, offs, ws, torch.cuda.current_stream())
            torch.cuda.synchronize()
            assert torch.equal(C.view(torch.int16), want.view(torch.int16))
        assert all(p.last_status() == B.GEMM_OK for p in plans)
    for p in plans:
        p.close()


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("kind", [B.GEMM_GROUPED_ROWS, B.GEMM_GROUPED_INNER])
def test_many_groups(kind, ctas):
    r = np.random.default_rng(3)
    counts = (r.integers(0, 9, 1024) * (r.random(1024) < 0.6)).tolist()
    R = int(np.sum(counts))
    A, Bm = _operands(kind, counts, R, 72, 136, "bf16", COL, 5)
    exact, absolute = _reference(kind, counts, R, 72, 136, COL, A, Bm)
    assert_rounded_sum(_run(kind, counts, 0, 72, 136, "bf16", COL, A, Bm, ctas=ctas), exact, absolute, 136)


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("kind", [B.GEMM_GROUPED_ROWS, B.GEMM_GROUPED_INNER])
def test_neighbours_do_not_leak(kind, ctas):
    """A group whose rows and matrix are NaN and infinite changes nothing in
    the groups beside it, at boundaries inside a tile."""
    counts, N, K = [37, 21, 70], 136, 200
    R = sum(counts)
    A, Bm = _operands(kind, counts, R, N, K, "f16", ROW, 9)
    clean = _run(kind, counts, 0, N, K, "f16", ROW, A, Bm, ctas=ctas)
    A[37:58] = float("nan")
    if kind == B.GEMM_GROUPED_ROWS:
        Bm[1] = float("inf")
    else:
        Bm[37:58] = float("inf")
    dirty = _run(kind, counts, 0, N, K, "f16", ROW, A, Bm, ctas=ctas)
    mine = slice(37, 58) if kind == B.GEMM_GROUPED_ROWS else slice(1, 2)
    assert bool(torch.isnan(dirty[mine]).all())
    clean[mine] = dirty[mine] = 0
    assert torch.equal(clean, dirty)


@pytest.mark.parametrize("kind", [B.GEMM_GROUPED_ROWS, B.GEMM_GROUPED_INNER])
def test_offsets_out_of_order_are_bounded(kind):
    """Offsets that fall, or pass the rows, are taken as the nearest in order
    and range."""
    counts, N, K = [10, 0, 30, 0], 64, 128
    R = 40
    A, Bm = _operands(kind, counts, R, N, K, "bf16", COL, 3)
    want = _run(kind, counts, 0, N, K, "bf16", COL, A, Bm)
    odd = torch.tensor([-5, 10, 4, 4000, 7], dtype=torch.int32, device="cuda")
    assert torch.equal(_run(kind, counts, 0, N, K, "bf16", COL, A, Bm, offsets=odd), want)


def test_new_offsets_streams_and_graphs_with_one_plan():
    """One plan and workspace, sizes that change from run to run, on a side
    stream and in a replayed graph."""
    E, R, N, K = 6, 300, 264, 512
    code, dt = DTYPES["bf16"]
    plan = B.GroupedPlan(B.GEMM_GROUPED_ROWS, E, R, N, K, code, COL)
    ws = torch.randint(0, 256, (max(1, plan.workspace_size),), dtype=torch.uint8, device="cuda")
    A, Bm = normal((R, K), dt, 1), normal((E, N, K), dt, 2, 0.25)
    C = torch.empty((R, N), dtype=dt, device="cuda")
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(A, Bm, C, offs, ws, torch.cuda.current_stream())
    for n, counts in enumerate(([50] * 6, [300, 0, 0, 0, 0, 0], [1, 2, 3, 0, 0, 290], [0] * 6, [17, 100, 33, 9, 1, 5])):
        fresh, _ = _sizes(counts)
        exact, absolute = _reference(B.GEMM_GROUPED_ROWS, counts, R, N, K, COL, A, Bm)
        for form in range(3):
            C.fill_(5)
            if form == 0:
                offs.copy_(fresh)
                plan.run(A, Bm, C, offs, ws, torch.cuda.current_stream())
            elif form == 1:
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    torch.cuda._sleep(5_000_000)
                    offs.copy_(fresh)
                    plan.run(A, Bm, C, offs, ws, side)
                side.synchronize()
            else:
                graph.replay()
            torch.cuda.synchronize()
            assert plan.last_status() == B.GEMM_OK
            assert_rounded_sum(C, exact, absolute, K, "sizes %d form %d" % (n, form))
    plan.close()


def test_matrices_past_32_bit_offsets():
    """The matrices together hold more than 2^32 elements; the last group's
    product is right."""
    E, N, K = 66, 8192, 8192  # 4.4e9 elements
    counts = [0] * E
    counts[0], counts[-2], counts[-1] = 3, 20, 9
    R = sum(counts)
    dt = torch.bfloat16
    A = normal((R, K), dt, 1)
    Bm = torch.zeros((E, N, K), dtype=dt, device="cuda")
    for e in (0, E - 2, E - 1):
        Bm[e] = normal((N, K), dt, e, 0.25)
    got = _run(B.GEMM_GROUPED_ROWS, counts, 0, N, K, "bf16", COL, A, Bm)
    at = 0
    for e in (0, E - 2, E - 1):
        n = counts[e]
        a, b = A[at:at + n].double(), Bm[e].double()
        assert_rounded_sum(got[at:at + n], a @ b.t(), a.abs() @ b.abs().t(), K)
        at += n


def test_gradients_against_differences():
    """L = <D, C(A, B)> is linear in A and in B: its difference quotient equals
    the gradients, which are the other two products, up to the output rounding
    of C (u of its magnitude) and of the gradient."""
    counts, N, K, dt = [9, 0, 30], 48, 64, torch.float16
    R = sum(counts)
    A, Bm = _operands(B.GEMM_GROUPED_ROWS, counts, R, N, K, "f16", ROW, 1)
    D = normal((R, N), dt, 5)
    # B is (E, K, N); the gradient to A is D B^T, the same memory as col-major N x K
    dA = _run(B.GEMM_GROUPED_ROWS, counts, 0, K, N, "f16", COL, D, Bm)
    dB = _run(B.GEMM_GROUPED_INNER, counts, 0, N, K, "f16", ROW, A, D)

    def loss(A, Bm):
        per = D.double() * _run(B.GEMM_GROUPED_ROWS, counts, 0, N, K, "f16", ROW, A, Bm).double()
        return per.sum().item(), per.abs().sum().item()

    u = 2.0 ** -11 + 2.0 ** -18

    def agree(value, plus, minus, h):
        (lp, mp), (lm, mm) = plus, minus
        assert abs((lp - lm) / h - value) <= u * (mp + mm) / h + u * abs(value)

    for r, k in ((0, 3), (8, 63), (9, 0), (38, 40)):
        ap, am = A.clone(), A.clone()
        ap[r, k] += 16
        am[r, k] -= 16
        agree(dA[r, k].item(), loss(ap, Bm), loss(am, Bm), (ap[r, k].double() - am[r, k].double()).item())
    for e, k, n in ((0, 5, 7), (2, 63, 47), (1, 2, 2)):
        bp, bm = Bm.clone(), Bm.clone()
        bp[e, k, n] += 16
        bm[e, k, n] -= 16
        agree(dB[e, k, n].item(), loss(A, bp), loss(A, bm), (bp[e, k, n].double() - bm[e, k, n].double()).item())


def test_empty_sizes_and_refusals():
    dt = torch.bfloat16
    offs = torch.zeros(4, dtype=torch.int32, device="cuda")
    C = Rows(1, 3 * 64 * 72, dt)
    with B.GroupedPlan(B.GEMM_GROUPED_ROWS, 3, 10, 64, 0, B.GEMM_BF16, COL) as p:  # nothing to sum: +0
        p.run(None, None, C, offs)
        assert bool((C.view[0, :640] == 0).all()) and bool((C.view[0, 640:] == 77).all())
    with B.GroupedPlan(B.GEMM_GROUPED_INNER, 3, 0, 64, 72, B.GEMM_BF16, COL) as p:
        p.run(None, None, C, offs)
        assert bool((C.view[0] == 0).all())
        C.check_guards()
    for kind, rows, N, K in ((0, 0, 64, 72), (0, 5, 0, 72), (1, 5, 0, 72), (1, 5, 64, 0)):
        with B.GroupedPlan(kind, 3, rows, N, K, B.GEMM_BF16, COL) as p:
            p.run(None, None, None, None)  # C is empty
    A, Bm = normal((10, 72), dt, 1), normal((3, 64, 72), dt, 2)
    with B.GroupedPlan(B.GEMM_GROUPED_ROWS, 3, 10, 64, 72, B.GEMM_BF16, COL) as p:
        ws = torch.empty(p.workspace_size, dtype=torch.uint8, device="cuda")
        good = [A, Bm, C, offs, ws]
        for i in range(5):
            for value, status in ((None, B.GEMM_ERR_WORKSPACE if i == 4 else B.GEMM_ERR_INVALID_ARG),
                                  (good[i].data_ptr() + 2, B.GEMM_ERR_WORKSPACE if i == 4 else B.GEMM_ERR_UNSUPPORTED)):
                args = list(good)
                args[i] = value
                with pytest.raises(B.GemmError) as e:
                    p.run(*args)
                assert e.value.status == status
        p.run(*good)
        assert p.last_status() == B.GEMM_OK
