"""Scaled products against their definition in 64 bits: every layout, type and
kind of scales, bit for bit on integers."""
import pytest
import torch

from moe_util import Rows
from persistent_stream_matmul_gb300 import _binding as B
from scaled_util import DTYPES, FP8, assert_product, operand_kind, product, scale_shape

pytestmark = pytest.mark.gpu

ROW, COL = B.GEMM_ROW_MAJOR, B.GEMM_COL_MAJOR
VEC, BLOCK = B.GEMM_SCALE_VECTOR, B.GEMM_SCALE_BLOCK


@pytest.fixture(scope="module", autouse=True)
def _ready():
    from gpu_util import ensure_built
    ensure_built()


def operand(rows, cols, type, kind, seed, integers):
    """A stored operand and its scales: normal values over the type's range, or whole numbers up to 3
    with scales that are powers of two."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = scale_shape(kind, rows, cols)
    if integers:
        v = torch.randint(-3, 4, (rows, cols), generator=g, device="cuda").float()
        s = torch.exp2(torch.randint(-2, 3, shape, generator=g, device="cuda").float())
    else:
        v = torch.randn(rows, cols, generator=g, device="cuda") * 40
        s = torch.exp(torch.randn(shape, generator=g, device="cuda"))
    return v.to(FP8[type][1]), s.contiguous()


class Case:
    def __init__(self, M, N, K, a="e4m3", b="e4m3", out="bf16", layout_a=ROW, layout_b=COL, scale_a=VEC, scale_b=BLOCK, seed=0,
                 integers=False, **options):
        self.M, self.N, self.K = M, N, K
        self.row_a, self.row_b = layout_a == ROW, layout_b == ROW
        self.kinds = operand_kind(scale_a, self.row_a), operand_kind(scale_b, not self.row_b)
        self.a, self.sa = operand(*((M, K) if self.row_a else (K, M)), a, self.kinds[0], seed, integers)
        self.b, self.sb = operand(*((K, N) if self.row_b else (N, K)), b, self.kinds[1], seed + 1, integers)
        self.code, self.dtype = DTYPES[out]
        self.plan = B.ScaledPlan(M, N, K, FP8[a][0], FP8[b][0], self.code, layout_a, layout_b, scale_a, scale_b, **options)
        self.ws = torch.full((max(16, self.plan.workspace_size),), 255, dtype=torch.uint8, device="cuda")

    def run(self, offset=0):
        C = Rows(self.M, self.N, self.dtype, None, offset)
        self.plan.run(self.a, self.sa, self.b, self.sb, C, self.ws)
        assert self.plan.last_status() == B.GEMM_OK
        C.check_guards()
        return C.view

    def reference(self):
        return product(self.a, self.sa, self.kinds[0], self.b, self.sb, self.kinds[1], self.row_a, self.row_b)

    def check(self, **kw):
        exact, absolute = self.reference()
        assert_product(self.run(**kw), exact, absolute, self.K)


FORWARD = dict(layout_a=ROW, layout_b=COL)
BACK = dict(layout_a=ROW, layout_b=ROW, a="e5m2")
WGRAD = dict(layout_a=COL, layout_b=ROW, a="e5m2", scale_b=VEC, out="f32")
TURNED = dict(layout_a=COL, layout_b=COL, b="e5m2", out="f16")

SIZES = [(1, 16, 16), (1, 128, 128), (1, 4096, 1024), (3, 208, 48), (16, 512, 2064), (17, 1040, 400), (33, 256, 4096), (96, 1024, 2048),
         (100, 16, 1040), (128, 128, 128), (129, 144, 272), (200, 4096, 512), (256, 256, 256), (257, 272, 144), (300, 1536, 2048),
         (512, 768, 1024), (640, 2304, 384), (1000, 1040, 2048)]


def sized(M, N, K, form):
    """The contiguous dimension of A rounded up to 16 where it is M."""
    return (M if form.get("layout_a", ROW) == ROW else -(-M // 16) * 16), N, K


@pytest.mark.parametrize("form", [FORWARD, BACK, WGRAD, TURNED], ids=["forward", "back", "wgrad", "turned"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, form):
    Case(*sized(M, N, K, form), seed=M + N + K, **form).check()


@pytest.mark.parametrize("options", [dict(form=B.GEMM_SCALED_TURNED), dict(form=B.GEMM_SCALED_STRAIGHT, ctas=1), dict(ctas=2),
                                     dict(form=B.GEMM_SCALED_FEW)], ids=["turned", "straight", "pairs", "few"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_in_every_form(M, N, K, options):
    Case(M, N, K, seed=M + N + K, **options).check()


@pytest.mark.parametrize("scale_a", [VEC, BLOCK])
@pytest.mark.parametrize("scale_b", [VEC, BLOCK])
@pytest.mark.parametrize("layout_a", [ROW, COL])
@pytest.mark.parametrize("layout_b", [ROW, COL])
@pytest.mark.parametrize("M,N,K", [(32, 272, 400), (272, 400, 656), (1, 400, 1040), (528, 544, 528)])
def test_integers_bit_for_bit(M, N, K, layout_a, layout_b, scale_a, scale_b):
    """Whole numbers up to 3 and scales 1/4 to 4: every partial sum is a multiple of 1/16 below 9 * 16 *
    1040 < 2^18, so it needs at most 22 bits and any order gives the same."""
    M = M if layout_a == ROW else -(-M // 16) * 16
    c = Case(M, N, K, out="f32", layout_a=layout_a, layout_b=layout_b, scale_a=scale_a, scale_b=scale_b, integers=True, seed=M)
    assert torch.equal(c.run().double(), c.reference()[0])


@pytest.mark.parametrize("a", FP8)
@pytest.mark.parametrize("b", FP8)
@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("M", [5, 300])
def test_types(a, b, out, M):
    c = Case(M, 272, 528, a, b, out, integers=True, seed=3)
    want = c.reference()[0]
    assert torch.equal(c.run(), want.float().to(c.dtype))  # exact in fp32, rounded once
    Case(M, 272, 528, a, b, out, seed=4).check()


@pytest.mark.parametrize("M,N", [(7, 33), (5, 1), (200, 333), (300, 1001), (257, 130)])
@pytest.mark.parametrize("out", DTYPES)
def test_rows_of_any_length_and_alignment(M, N, out):
    for options in (dict(form=B.GEMM_SCALED_FEW), dict(form=B.GEMM_SCALED_TURNED), dict(form=B.GEMM_SCALED_STRAIGHT, ctas=1), dict(ctas=2)):
        for offset in (0, 1, 4):
            Case(M, N, 272, out=out, seed=N, **options).check(offset=offset)


@pytest.mark.parametrize("K", [0, 16, 112, 128, 144, 256, 272])
@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("options", [{}, dict(form=B.GEMM_SCALED_TURNED), dict(form=B.GEMM_SCALED_STRAIGHT), dict(ctas=2)])
def test_short_sums(M, K, options):
    c = Case(M, 256, K, seed=K, **options)
    if K == 0:
        assert not c.run().any() and not torch.signbit(c.run()).any()
    else:
        c.check()


@pytest.mark.parametrize("options", [{}, dict(form=B.GEMM_SCALED_TURNED), dict(form=B.GEMM_SCALED_STRAIGHT), dict(ctas=2)])
def test_nan_and_infinity_stay_in_their_row_and_column(options):
    for M in (20, 400):
        c = Case(M, 400, 400, seed=M, **options)
        a = c.a.float()
        a[3, 7] = float("nan")
        c.a.copy_(a.to(c.a.dtype))
        c.sa[1, 11] = float("inf")   # group 1 of row 11
        c.sb[2, 0] = float("nan")    # columns 256 .. 383, group 0
        got = c.run()
        bad = torch.zeros(M, 400, dtype=torch.bool, device="cuda")
        bad[3], bad[11], bad[:, 256:384] = True, True, True
        assert torch.equal(~torch.isfinite(got), bad)


def test_repeats_bitwise_and_workspace_of_another_plan():
    """One workspace for plans that leave different things in it, and a captured run beside them."""
    cases = [Case(96, 1024, 8192, seed=1), Case(640, 1280, 2048, seed=2), Case(1, 2048, 4096, seed=3)]
    ws = torch.full((max(c.ws.numel() for c in cases),), 255, dtype=torch.uint8, device="cuda")
    for c in cases:
        c.ws = ws
    first = [c.run().clone() for c in cases]
    for c, f in zip(cases, first):
        exact, absolute = c.reference()
        assert_product(f, exact, absolute, c.K)
    graph, outs = torch.cuda.CUDAGraph(), [torch.empty_like(f) for f in first]
    with torch.cuda.graph(graph):
        for c, o in zip(cases, outs):
            c.plan.run(c.a, c.sa, c.b, c.sb, o, ws, torch.cuda.current_stream())
    for _ in range(4):
        for o in outs:
            o.zero_()
        graph.replay()
        assert all(torch.equal(o, f) for o, f in zip(outs, first))
        assert all(torch.equal(c.run(), f) for c, f in zip(cases, first))


def test_quantised_layer_end_to_end():
    """norm -> product -> gradients, as a program runs them: each product within its bound for the
    operands that the quantisation made."""
    T, H, F = 200, 272, 400
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, w = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(3))
    W = torch.randn(F, H, generator=g, device="cuda").bfloat16()
    dy = torch.randn(T, F, generator=g, device="cuda").bfloat16()

    def empty(rows, cols, kind, type="e4m3"):
        return torch.empty(rows, cols, dtype=FP8[type][1], device="cuda"), torch.empty(scale_shape(kind, rows, cols), device="cuda")

    s, y = torch.empty_like(x), torch.empty_like(x)
    q, qs = empty(T, H, "rows")
    B.gemm_rms_norm(x, H, r, H, w[0], 1e-5, T, H, B.GEMM_BF16, s, H, y, H, q, H, 0, qs, None)
    Wq, Ws = empty(F, H, "blocks")
    B.gemm_scaled_quantize(B.GEMM_QUANTIZE_BLOCKS, W, H, F, H, B.GEMM_BF16, 0, Wq, H, Ws)
    yq, ys = empty(T, H, "cols")
    B.gemm_scaled_quantize(B.GEMM_QUANTIZE_COLS, y, H, T, H, B.GEMM_BF16, 0, yq, H, ys)
    dr, drs = empty(T, F, "rows", "e5m2")
    dc, dcs = empty(T, F, "cols", "e5m2")
    B.gemm_scaled_quantize_both(dy, F, T, F, B.GEMM_BF16, 1, dr, F, drs, dc, F, dcs)
    for M, N, K, A, sa, ka, ta, la, Bm, sb, kb, lb, scale_b in (
            (T, F, H, q, qs, "rows", 0, ROW, Wq, Ws, "blocks", COL, BLOCK), (T, H, F, dr, drs, "rows", 1, ROW, Wq, Ws, "blocks", ROW, BLOCK),
            (F, H, T, dc, dcs, "cols", 1, COL, yq, ys, "cols", ROW, VEC)):
        p = B.ScaledPlan(M, N, K, ta, 0, B.GEMM_BF16, la, lb, VEC, scale_b)
        C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(16, p.workspace_size), dtype=torch.uint8, device="cuda")
        p.run(A, sa, Bm, sb, C, ws)
        assert p.last_status() == B.GEMM_OK
        assert_product(C, *product(A, sa, ka, Bm, sb, kb, la == ROW, lb == ROW), K)


# every form of the kernel on tensor memory, whatever the plan would choose: (ctas, form)
FORMS = [(1, B.GEMM_SCALED_STRAIGHT), (2, B.GEMM_SCALED_STRAIGHT), (1, B.GEMM_SCALED_TURNED)]


@pytest.mark.parametrize("ctas,form", FORMS)
@pytest.mark.parametrize("layout_a", [ROW, COL])
@pytest.mark.parametrize("layout_b", [ROW, COL])
@pytest.mark.parametrize("scale_a,scale_b", [(VEC, BLOCK), (VEC, VEC), (BLOCK, VEC), (BLOCK, BLOCK)])
@pytest.mark.parametrize("M,N,K", [(16, 144, 272), (304, 528, 784), (528, 272, 4112)])
def test_forms(M, N, K, layout_a, layout_b, scale_a, scale_b, ctas, form):
    kw = dict(layout_a=layout_a, layout_b=layout_b, scale_a=scale_a, scale_b=scale_b, ctas=ctas, form=form)
    for out in ("f32", "bf16"):
        Case(M, N, K, out=out, seed=M, **kw).check()
    c = Case(M, N, K, out="f32", integers=True, seed=M, **kw)
    assert c.plan.info("ctas") == ctas and c.plan.info("form") == form
    # whole sixteenths below 9 * 16 * 4112 < 2^20: 24 bits, exact in any order
    assert torch.equal(c.run().double(), c.reference()[0])


@pytest.mark.parametrize("ctas,form,M,N,K", [(2, 0, 2048, 2560, 4096), (2, 0, 512, 512, 16384), (1, 0, 1280, 2048, 2304),
                                               (1, 0, 128, 128, 20000), (1, 1, 48, 512, 8192), (1, 1, 300, 8192, 4096), (1, 1, 1, 128, 65536)])
@pytest.mark.parametrize("scale_b", [VEC, BLOCK])
def test_split_tiles(ctas, form, M, N, K, scale_b):
    """Tiles left over a whole round of the units, or fewer than one, cut along k and joined."""
    c = Case(M, N, K, out="f32", integers=False, seed=K, ctas=ctas, form=form, scale_b=scale_b)
    assert c.plan.info("shares") > 1
    first = c.run().clone()
    exact, absolute = c.reference()
    assert_product(first, exact, absolute, K)
    for _ in range(5):
        assert torch.equal(c.run(), first)


@pytest.mark.parametrize("ctas,form", FORMS)
def test_timeout_is_reported_and_replays_recover(ctas, form):
    c = Case(96, 1024, 8192, seed=5, ctas=ctas, form=form)
    want = c.run().clone()
    out, graph, stream = torch.empty_like(want), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        c.plan.run(c.a, c.sa, c.b, c.sb, out, c.ws, stream)
    with torch.cuda.stream(stream):
        for unit in (0, 3):
            c.plan.set_option(B.GEMM_SCALED_OPT_INJECT_GIVE_UP, unit)
            graph.replay()
            assert c.plan.last_status(stream) == B.GEMM_ERR_TIMEOUT
            assert c.plan.last_status(stream) == B.GEMM_OK
            c.plan.set_option(B.GEMM_SCALED_OPT_INJECT_GIVE_UP, -1)
            for _ in range(3):
                out.fill_(7)
                graph.replay()
                assert c.plan.last_status(stream) == B.GEMM_OK
                assert torch.equal(out, want)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 24, 25, 32, 33, 70, 129])
@pytest.mark.parametrize("N,K", [(1, 16), (17, 128), (33, 144), (4096, 2064), (9999, 1040), (500, 14336)])
@pytest.mark.parametrize("scale_a,scale_b", [(VEC, BLOCK), (VEC, VEC), (BLOCK, VEC)])
def test_few_rows(M, N, K, scale_a, scale_b):
    few = dict(scale_a=scale_a, scale_b=scale_b, form=B.GEMM_SCALED_FEW)
    c = Case(M, N, K, seed=M + N, **few)
    assert c.plan.info("form") == B.GEMM_SCALED_FEW and c.plan.workspace_size == 0
    c.check()
    Case(M, N, K, "e5m2", "e4m3", "f32", seed=N, **few).check(offset=1)
    c = Case(M, N, K, out="f32", integers=True, seed=M, **few)
    assert torch.equal(c.run().double(), c.reference()[0])  # sixteenths below 9 * 16 * 14336 < 2^21: 25 bits at most


@pytest.mark.parametrize("K", [1, 3, 127, 129, 1000])
@pytest.mark.parametrize("M,N", [(16, 16), (48, 400), (400, 272), (4112, 4096)])
def test_sums_over_any_number_of_tokens(M, N, K):
    """Both operands MN-major: the summed dimension needs no alignment."""
    Case(M, N, K, seed=K, **WGRAD).check()
    c = Case(M, N, K, out="f32", layout_a=COL, layout_b=ROW, scale_b=VEC, integers=True, seed=K)
    assert torch.equal(c.run().double(), c.reference()[0])


@pytest.mark.parametrize("M", [3, 24, 200])
def test_offsets_past_32_bits(M):
    """B of 2.3 GB: its last rows against 64 bits, and its first, in each form."""
    N, K = 140016, 16384
    g = torch.Generator(device="cuda").manual_seed(M)
    a = (torch.randn(M, K, generator=g, device="cuda") * 20).to(torch.float8_e4m3fn)
    some = (torch.randn(1008, K, generator=g, device="cuda") * 20).to(torch.float8_e4m3fn)
    b = torch.empty(N, K, dtype=torch.uint8, device="cuda")
    b[:1008] = some.view(torch.uint8)
    for at in range(1008, N, 1008):
        b[at:at + 1008] = b[:min(1008, N - at)]
    sa = torch.exp(torch.randn(K // 128, M, generator=g, device="cuda"))
    sb = torch.exp(torch.randn(K // 128, N, generator=g, device="cuda"))
    p = B.ScaledPlan(M, N, K, 0, 0, B.GEMM_F32, ROW, COL, VEC, VEC)
    assert p.info("form") == {3: B.GEMM_SCALED_FEW, 24: B.GEMM_SCALED_TURNED, 200: B.GEMM_SCALED_STRAIGHT}[M]
    ws = torch.empty(max(16, p.workspace_size), dtype=torch.uint8, device="cuda")
    C = torch.empty(M, N, device="cuda")
    p.run(a, sa, b, sb, C, ws)
    assert p.last_status() == B.GEMM_OK
    for rows in (slice(0, 300), slice(N - 300, N)):
        part = b[rows].contiguous().view(torch.float8_e4m3fn)
        assert_product(C[:, rows], *product(a, sa, "rows", part, sb[:, rows].contiguous(), "rows", True, False), K)


def test_device_of_the_plan_is_kept():
    before = torch.cuda.current_device()
    c = Case(300, 272, 272, seed=1)
    c.check()
    assert torch.cuda.current_device() == before
