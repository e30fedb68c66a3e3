"""Helpers shared by the tests of the mixture-of-experts operators: routings,
guarded device buffers, 64-bit references and derived error bounds."""
import numpy as np
import torch

from persistent_stream_matmul_gb300 import _binding as B

DTYPES = {"bf16": (B.GEMM_BF16, torch.bfloat16), "f16": (B.GEMM_F16, torch.float16)}
# unit roundoff of the output type, and half its smallest subnormal
ROUNDOFF = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25)}
SENTINEL = 77


def routing(tokens, topk, experts, seed, drop=0.0, skew=0.0):
    """Choices (tokens, topk) int64 with dropped slots of several kinds."""
    r = np.random.default_rng(seed)
    p = (1.0 + np.arange(experts)) ** -skew
    ids = r.choice(experts, size=(tokens, topk), p=p / p.sum()).astype(np.int64)
    bad = r.choice(np.array([-1, -7, experts, experts + 5, 2 ** 31 - 1, -2 ** 31]), size=ids.shape)
    return np.where(r.random(ids.shape) < drop, bad, ids)


def sorted_slots(ids, experts):
    """(offsets, rows, slots) of the stable sort, slot by slot."""
    flat = ids.reshape(-1)
    by = [[] for _ in range(experts)]
    for s, e in enumerate(flat.tolist()):
        if 0 <= e < experts:
            by[e].append(s)
    offsets = np.concatenate([[0], np.cumsum([len(b) for b in by])]).astype(np.int32)
    slots = np.full(flat.size, -1, dtype=np.int32)
    rows = np.full(flat.size, -1, dtype=np.int32)
    order = [s for b in by for s in b]
    slots[:len(order)] = order
    rows[order] = np.arange(len(order))
    return offsets, rows, slots


class Rows:
    """A rows x cols device matrix with a leading dimension, an element offset
    from the allocation's (aligned) start, and sentinels around every row."""

    def __init__(self, rows, cols, dtype, ld=None, offset=0):
        self.rows, self.cols, self.ld = rows, cols, ld or cols
        self.buf = torch.full((offset + rows * self.ld + 64,), SENTINEL, dtype=dtype, device="cuda")
        self.offset = offset
        self.view = torch.as_strided(self.buf, (rows, cols), (self.ld, 1), offset)

    def data_ptr(self):
        return self.buf.data_ptr() + self.offset * self.buf.element_size()

    def set(self, values):
        self.view.copy_(values)
        return self

    def check_guards(self):
        keep = torch.ones_like(self.buf, dtype=torch.bool)
        torch.as_strided(keep, (self.rows, self.cols), (self.ld, 1), self.offset).fill_(False)
        assert bool((self.buf[keep] == SENTINEL).all()), "write outside the rows"


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def assert_rounded_sum(got, exact, absolute, terms, note=""):
    """`got` (16-bit) is `exact` after an fp32 sum of `terms` products with sum
    of magnitudes `absolute`, rounded once: an fp32 sum of n terms in any order
    is within n * 2^-24 / (1 - n * 2^-24) of the magnitudes when each addition
    rounds to nearest, twice that when it truncates; the products of 16-bit
    values are exact in fp32 and a weight adds one rounding, counted as one
    more term.  The output rounding adds u * |value| (or half a subnormal)."""
    u, tiny = ROUNDOFF[got.dtype]
    e = (terms + 1) * 2.0 ** -23 * absolute * 1.01
    bound = e + u * (exact.abs() + e) + tiny
    err = (got.double() - exact).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), "%s: %d values out of bound, worst %.3g of it" % (
        note, int(bad.sum()), float((err / bound.clamp(min=1e-300)).max()))
