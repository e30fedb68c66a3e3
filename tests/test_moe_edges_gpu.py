"""GPU tests of the mixture-of-experts operators at their edges."""
import threading

import numpy as np
import pytest
import torch

from persistent_stream_matmul_gb300 import _binding as B
from tests.gpu_util import ensure_built
from tests.moe_util import DTYPES, Rows, assert_rounded_sum, normal, routing, sorted_slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("kind", [B.GEMM_GROUPED_ROWS, B.GEMM_GROUPED_INNER])
@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("first,counts,unused,N,K", [(11, [9, 13], 7, 64, 128), (1, [0, 0], 5, 72, 200), (300, [40], 0, 520, 2304),
                                                     (5000, [0, 700, 3], 300, 264, 64), (17, [0], 0, 8, 8)])
def test_offsets_that_start_inside_the_rows(first, counts, unused, N, K, ctas, kind):
    """The rows before the first group are unused: +0 in ROWS, and whatever
    they hold, in no sum."""
    code, dt = DTYPES["bf16"]
    R, G, rows = first + sum(counts) + unused, len(counts), kind == B.GEMM_GROUPED_ROWS
    offsets = first + np.concatenate([[0], np.cumsum(counts)])
    A, Bm = normal((R, K), dt, 1), normal((G, K, N) if rows else (R, N), dt, 2, 0.25)
    for used in ([A] if rows else [A, Bm]):
        used[:first] = float("nan")
        used[first + sum(counts):] = float("nan")
    C = Rows(R if rows else G * K, N, dt, offset=64)
    with B.GroupedPlan(kind, G, R, N, K, code, B.GEMM_ROW_MAJOR, ctas=ctas) as p:
        ws = torch.empty(max(1, p.workspace_size), dtype=torch.uint8, device="cuda")
        p.run(A, Bm, C, torch.tensor(offsets, dtype=torch.int32, device="cuda"), ws)
        assert p.last_status() == B.GEMM_OK
    C.check_guards()
    exact = torch.zeros(C.view.shape, dtype=torch.float64, device="cuda")
    absolute = torch.zeros_like(exact)
    for g, n in enumerate(counts):
        at = slice(offsets[g], offsets[g + 1])
        a, b = A[at].double(), (Bm[g] if rows else Bm[at]).double()
        out = at if rows else slice(g * K, (g + 1) * K)
        a = a if rows else a.t()
        exact[out], absolute[out] = a @ b, a.abs() @ b.abs()
    assert_rounded_sum(C.view, exact, absolute, K if rows else max(1, max(counts)))
    if rows:
        unused_rows = torch.cat([C.view[:first], C.view[first + sum(counts):]])
        assert not bool(unused_rows.view(torch.int16).any())  # +0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,ld", [(1, 1, 0), (5, 2, 1), (40, 3, 3), (1500, 2, 1), (300, 9, 8)])
def test_gradient_of_combine_without_elements(T, k, ld, dtype):
    """hidden == 0: no row has an element to read, at NULL or at any address;
    the weights' gradients are empty sums."""
    code, dt = DTYPES[dtype]
    rows = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).contiguous()
    rows[::3] = -1
    slots = torch.arange(T * k, dtype=torch.int32, device="cuda")
    w = torch.rand(T * k, device="cuda")
    few = Rows(1, 8, dt, offset=1)  # a row of no elements may start off a boundary
    for p in (None, few):
        dw = Rows(1, T * k, torch.float32)
        B.gemm_moe_combine_grad(p, ld, p, ld, rows, slots, w, T, k, 0, code, p, ld, dw)
        torch.cuda.synchronize()
        assert not bool(dw.view.view(torch.int32).any())  # +0
        dw.check_guards()
    assert bool((few.buf == 77).all())


@pytest.mark.parametrize("ctas", [1, 2])
def test_rows_up_to_the_largest_index(ctas):
    """One group of 2 140 000 000 rows and the rest in another: every row of C,
    whole numbers, so exactly."""
    R, N, K = 2 ** 31 - 1024, 8, 8
    dt, step = torch.bfloat16, 2 ** 25
    A = torch.empty((R, K), dtype=dt, device="cuda")  # 34 GB, and as much for C
    for at in range(0, R, step):
        part = A[at:at + step].view(torch.int16)
        torch.randint(0, 16, part.shape, out=part, dtype=torch.int16, device="cuda")
        A[at:at + step] = part.to(dt) - 8
    Bm = torch.randint(-2, 3, (2, K, N), device="cuda").to(dt)
    C = torch.full((R, N), 7, dtype=dt, device="cuda")
    offsets = [3, 2_140_000_000, R]
    with B.GroupedPlan(B.GEMM_GROUPED_ROWS, 2, R, N, K, B.GEMM_BF16, B.GEMM_ROW_MAJOR, ctas=ctas) as p:
        ws = torch.empty(max(1, p.workspace_size), dtype=torch.uint8, device="cuda")
        p.run(A, Bm, C, torch.tensor(offsets, dtype=torch.int32, device="cuda"), ws, torch.cuda.current_stream())
        assert p.last_status(torch.cuda.current_stream()) == B.GEMM_OK
    assert not bool(C[:3].view(torch.int16).any())
    for g in range(2):
        for at in range(offsets[g], offsets[g + 1], step):
            end = min(at + step, offsets[g + 1])
            assert torch.equal(C[at:end], (A[at:end].float() @ Bm[g].float()).to(dt)), at


@pytest.mark.parametrize("layout", [B.GEMM_COL_MAJOR, B.GEMM_ROW_MAJOR])
@pytest.mark.parametrize("ctas", [1, 2])
def test_blocks_that_end_inside_a_step(ctas, layout):
    """Groups of every size from 1 to 63 and beyond, each followed by one of NaN
    and infinite rows: the rows past a group's end that its last block covers add
    nothing, in either CTA of a pair, run after run."""
    counts = [n for i in range(1, 130) for n in (i, 1 + i % 3)]
    R, G, N, K = sum(counts) + 5, len(counts), 328, 264
    offsets = np.concatenate([[0], np.cumsum(counts)])
    g = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randint(-2, 3, (R, K), generator=g, device="cuda").half()
    D = torch.randint(-2, 3, (R, N), generator=g, device="cuda").half()
    want = torch.zeros((G, K, N), dtype=torch.float64, device="cuda")
    for e in range(0, G, 2):
        at = slice(offsets[e], offsets[e + 1])
        want[e] = A[at].double().t() @ D[at].double()
        A[offsets[e + 1]:offsets[e + 2]] = float("nan")
        D[offsets[e + 1]:offsets[e + 2]] = float("inf")
    A[offsets[-1]:] = D[offsets[-1]:] = float("nan")
    want = want[::2].transpose(1, 2) if layout == B.GEMM_COL_MAJOR else want[::2]
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    C = torch.empty((G, *want.shape[1:]), dtype=torch.float16, device="cuda")
    with B.GroupedPlan(B.GEMM_GROUPED_INNER, G, R, N, K, B.GEMM_F16, layout, ctas=ctas) as p:
        ws = torch.empty(max(1, p.workspace_size), dtype=torch.uint8, device="cuda")
        for _ in range(10):
            C.fill_(7)
            p.run(A, D, C, offs, ws, torch.cuda.current_stream())
            assert torch.equal(C[::2].double(), want)  # whole numbers, at most 4 * 129
            assert bool(torch.isnan(C[1::2]).all())
        assert p.last_status(torch.cuda.current_stream()) == B.GEMM_OK


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("kind", [B.GEMM_GROUPED_ROWS, B.GEMM_GROUPED_INNER])
def test_replays_after_a_timeout(kind, ctas):
    """A captured launch in which one contributor to a split tile gives up: the
    timeout is reported, and the next replays join what they themselves summed,
    which leaves every counter (the workspace's first words, one a CTA) at none."""
    counts, N, K = ([2, 0, 5], 72, 8192) if kind == B.GEMM_GROUPED_ROWS else ([700, 8300, 0], 72, 136)
    G, R = len(counts), sum(counts)
    code, dt = DTYPES["bf16"]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    Bm = normal((G, N, K) if kind == B.GEMM_GROUPED_ROWS else (R, N), dt, 2, 0.25)
    A = torch.empty((R, K), dtype=dt, device="cuda")
    C = torch.empty((R, N) if kind == B.GEMM_GROUPED_ROWS else (G, N, K), dtype=dt, device="cuda")
    p = B.GroupedPlan(kind, G, R, N, K, code, B.GEMM_COL_MAJOR, ctas=ctas)
    work = {u: p.units(offsets, u) for u in range(p.info("units"))}
    split = [u for u, w in work.items() if w and w[0][0] < 0]
    assert len(split) > 3 and max(len(w) for w in work.values()) == 1
    ws = torch.zeros(p.workspace_size, dtype=torch.uint8, device="cuda")
    counts_in = ws[:8 * p.info("units") * ctas].view(torch.int64)
    stream = torch.cuda.current_stream()
    A.copy_(normal((R, K), dt, 1))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(A, Bm, C, offs, ws, torch.cuda.current_stream())
    for n, unit in enumerate((split[0], split[-1], split[len(split) // 2])):
        p.set_option(B.GEMM_GROUPED_OPT_INJECT_GIVE_UP, unit)
        for _ in range(n):
            graph.replay()
        graph.replay()
        assert p.last_status(stream) == B.GEMM_ERR_TIMEOUT
        assert p.last_status(stream) == B.GEMM_OK
        p.set_option(B.GEMM_GROUPED_OPT_INJECT_GIVE_UP, -1)
        for again in range(3):
            A.copy_(normal((R, K), dt, 10 * n + again))  # what the run before left is wrong now
            want = torch.empty_like(C)
            p.run(A, Bm, want, offs, torch.zeros_like(ws), stream)
            C.fill_(7)
            graph.replay()
            assert p.last_status(stream) == B.GEMM_OK
            assert torch.equal(C.view(torch.int16), want.view(torch.int16))
            assert not bool((counts_in & 0xffff).any())
    p.close()


@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,E", [(131072, 8, 64), (131073, 8, 256), (300001, 5, 1000), (1200003, 1, 3), (2 ** 22 + 1, 4, 1024)])
def test_sorts_of_more_than_a_million_slots(T, k, E, id_type):
    """From 1048577 slots on a warp takes its part in several batches, the last
    block's some in one and some in none."""
    g = torch.Generator(device="cuda").manual_seed(T)
    n, pad = T * k, 3
    ids = (torch.rand((T, k + pad), generator=g, device="cuda") ** 3 * E).to(id_type).clamp_(max=E - 1)
    ids[torch.rand((T, k + pad), generator=g, device="cuda") < 0.1] = -1
    ids[::7, 0] = E
    key = ids[:, :k].reshape(-1).long()
    kept = (key >= 0) & (key < E)
    order = torch.sort(torch.where(kept, key, E), stable=True).indices
    total = int(kept.sum())
    counts = torch.bincount(key[kept], minlength=E)
    offsets, rows, slots = (Rows(1, m, torch.int32) for m in (E + 1, n, n))
    ws = torch.randint(0, 256, (B.gemm_moe_sort_workspace_size(T, k, E),), dtype=torch.uint8, device="cuda")
    B.gemm_moe_sort(ids, B.GEMM_INDEX_I64 if id_type == torch.int64 else B.GEMM_INDEX_I32, k + pad, T, k, E,
                    offsets, rows, slots, ws, torch.cuda.current_stream())
    assert torch.equal(offsets.view[0, 1:].long(), counts.cumsum(0)) and int(offsets.view[0, 0]) == 0
    assert torch.equal(slots.view[0, :total].long(), order[:total]) and bool((slots.view[0, total:] == -1).all())
    want = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    want[order[:total]] = torch.arange(total, device="cuda")
    assert torch.equal(rows.view[0].long(), want)
    for o in (offsets, rows, slots):
        o.check_guards()


def test_sorts_of_two_threads_do_not_disturb_each_other():
    """Sorts of different numbers of experts, and so of shared memory, on two
    host threads with a stream each."""
    T, k = 2000, 2
    failures = []

    def work(experts, seed, calls):
        try:
            ids = routing(T, k, experts, seed)
            want = sorted_slots(ids, experts)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                dev = torch.from_numpy(ids).cuda()
                out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (experts + 1, T * k, T * k)]
            for _ in range(calls):
                B.gemm_moe_sort(dev, B.GEMM_INDEX_I64, k, T, k, experts, *out, None, stream)
            stream.synchronize()
            for got, w in zip(out, want):
                assert np.array_equal(got.cpu().numpy(), w)
        except BaseException as e:
            failures.append(e)

    assert B.gemm_moe_sort_workspace_size(T, k, 1024) == 0
    threads = [threading.Thread(target=work, args=(e, e, 5000)) for e in (300, 1024, 400, 1000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[0]
