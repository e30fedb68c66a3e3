"""Helpers shared by the tests of the 8-bit linear layer: 64-bit definitions of
its operators, written from their formulas, and derived error bounds."""
import torch

from persistent_stream_matmul_gb300 import _binding as B

DTYPES = {"bf16": (B.GEMM_BF16, torch.bfloat16), "f16": (B.GEMM_F16, torch.float16), "f32": (B.GEMM_F32, torch.float32)}
FP8 = {"e4m3": (B.GEMM_E4M3, torch.float8_e4m3fn, 448.0, 3, -6), "e5m2": (B.GEMM_E5M2, torch.float8_e5m2, 57344.0, 2, -14)}
KINDS = {"rows": B.GEMM_QUANTIZE_ROWS, "cols": B.GEMM_QUANTIZE_COLS, "blocks": B.GEMM_QUANTIZE_BLOCKS}
# unit roundoff of the output type, and half its smallest subnormal
ROUNDOFF = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25), torch.float32: (2.0 ** -24, 2.0 ** -150)}
GROUP = 128
LEAST = 2.0 ** -100


def up(n):
    return -(-n // GROUP)


def scale_shape(kind, rows, cols):
    return {"rows": (up(cols), rows), "cols": (up(rows), cols), "blocks": (up(rows), up(cols))}[kind]


def magnitudes(x, kind):
    """The largest magnitude of every group of a 64-bit matrix, in the order of its scales."""
    rows, cols = x.shape
    big = torch.zeros(up(rows) * GROUP, up(cols) * GROUP, dtype=torch.float64, device=x.device)
    big[:rows, :cols] = torch.where(torch.isnan(x), 0.0, x.abs())
    big = big.view(up(rows), GROUP, up(cols), GROUP)
    m = {"rows": lambda: big.amax(3).reshape(-1, up(cols))[:rows].t(), "cols": lambda: big.amax(1).reshape(up(rows), -1)[:, :cols],
         "blocks": lambda: big.amax(3).amax(1)}[kind]()
    return m.clamp(min=LEAST)


def spread(table, rows, cols, kind):
    """The entry of a table in the order of the scales for every element."""
    r = torch.arange(rows, device=table.device) // (1 if kind == "rows" else GROUP)
    c = torch.arange(cols, device=table.device) // (1 if kind == "cols" else GROUP)
    return (table.t() if kind == "rows" else table)[r][:, c]


def to_grid(v, type):
    """The nearest 8-bit values of 64-bit ones, ties to an even last digit."""
    _, _, _, digits, least = FP8[type]
    exponent = (torch.frexp(v).exponent.long() - 1).clamp(min=least) - digits
    step = ((exponent + 1023) << 52).view(torch.float64)  # 2 to that power, exactly
    return torch.round(v / step) * step


def quantized(x, type, kind):
    """(values, scales) of a 64-bit matrix by the definition; the scales not yet rounded to fp32."""
    m, largest = magnitudes(x, kind), FP8[type][2]
    return to_grid(x * largest / spread(m, *x.shape, kind), type), m / largest


def activations(shape, dtype, seed, spread_by=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp(spread_by * torch.randn(shape[0], 1, generator=g, device="cuda"))).to(dtype)


def operand_kind(scale, contiguous_k):
    """Which elements of a stored operand share a scale."""
    return "blocks" if scale == B.GEMM_SCALE_BLOCK else "rows" if contiguous_k else "cols"


def product(a, sa, ka, b, sb, kb, row_a, row_b):
    """C and the sum of magnitudes in 64 bits, of stored 8-bit operands."""
    A = a.float().double() * spread(sa.double(), *a.shape, ka)
    Bm = b.float().double() * spread(sb.double(), *b.shape, kb)
    A, Bm = A if row_a else A.t(), Bm if row_b else Bm.t()
    return A @ Bm, A.abs() @ Bm.abs()


def assert_product(got, exact, absolute, K, note=""):
    """`got` is `exact` within the order of its sums: K exact products (of 4 by 4 bits) are added in
    fp32, 128 at a time, each addition within 2^-23 of the magnitudes even if it truncates; a group's sum
    takes up to three more roundings (two scales and the addition), and the result one to its type."""
    u, tiny = ROUNDOFF[got.dtype]
    e = (min(K, 128) + 3 * up(K) + 3) * 2.0 ** -23 * absolute * 1.01
    bound = e + u * (exact.abs() + e) + tiny
    err = (got.double() - exact).abs()
    # past the largest value (and half its step) the result is infinite
    over = {torch.float16: 65520.0, torch.bfloat16: (2 - 2.0 ** -8) * 2.0 ** 127, torch.float32: (2 - 2.0 ** -24) * 2.0 ** 127}[got.dtype]
    err = torch.where((got == torch.sign(exact) * float("inf")) & (exact.abs() + e >= over), 0.0, err)
    bad = ~(err <= bound)
    assert not bool(bad.any()), "%s: %d values out of bound, worst %.3g of it" % (
        note, int(bad.sum()), float((err / bound.clamp(min=1e-300)).max()))
