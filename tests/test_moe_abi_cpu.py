"""Refusals of the mixture-of-experts entry points.  They come before any
device call, so they need no GPU; the operands are addresses that are never
read."""
import ctypes

import pytest

from persistent_stream_matmul_gb300 import _binding as B
from persistent_stream_matmul_gb300 import build

P = 0x1000  # an aligned address
INV, UNS = B.GEMM_ERR_INVALID_ARG, B.GEMM_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    B.load()


def refused(status, fn, *args):
    with pytest.raises(B.GemmError) as e:
        fn(*args)
    assert e.value.status == status, e.value


def _with(base, **changes):
    return [changes.get(k, v) for k, v in base.items()]


SORT = dict(ids=P, id_type=1, ld=2, tokens=4, topk=2, experts=8, offsets=P, rows=P, slots=P, ws=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INV, dict(ids=None)), (INV, dict(offsets=None)), (INV, dict(rows=None)), (INV, dict(slots=None)),
    (INV, dict(id_type=2)), (INV, dict(id_type=-1)), (INV, dict(ld=1)), (INV, dict(tokens=-1)), (INV, dict(topk=0)),
    (INV, dict(experts=0)), (UNS, dict(experts=1025)), (UNS, dict(tokens=2 ** 30)), (UNS, dict(tokens=2 ** 62)), (UNS, dict(topk=65536, ld=65536)),
    (UNS, dict(ids=P + 4)), (UNS, dict(ids=P + 2, id_type=0)), (UNS, dict(offsets=P + 2)), (UNS, dict(rows=P + 1)),
    (UNS, dict(slots=P + 2))])
def test_sort_refusals(status, changes):
    refused(status, B.gemm_moe_sort, *_with(SORT, **changes))


def test_sort_workspace_size():
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 2, 0)):
        refused(INV, B.gemm_moe_sort_workspace_size, *bad)
    refused(UNS, B.gemm_moe_sort_workspace_size, 4, 2, 1025)
    refused(UNS, B.gemm_moe_sort_workspace_size, 2 ** 40, 2, 8)
    assert B.load().gemm_moe_sort_workspace_size(4, 2, 8, None) == INV
    assert B.gemm_moe_sort_workspace_size(0, 1, 1) >= 0
    big = B.gemm_moe_sort_workspace_size(32768, 8, 256)
    if big:
        refused(B.GEMM_ERR_WORKSPACE, B.gemm_moe_sort, *_with(SORT, tokens=32768, topk=8, ld=8, experts=256, ws=None))
        refused(B.GEMM_ERR_WORKSPACE, B.gemm_moe_sort, *_with(SORT, tokens=32768, topk=8, ld=8, experts=256, ws=P + 8))


DISPATCH = dict(x=P, ldx=16, rows=P, slots=P, tokens=4, topk=2, hidden=16, dtype=1, xs=P, ldxs=16, stream=None)
DISPATCH_GRAD = dict(dxs=P, lddxs=16, rows=P, tokens=4, topk=2, hidden=16, dtype=1, dx=P, lddx=16, stream=None)
COMBINE = dict(ys=P, ldys=16, rows=P, weights=P, tokens=4, topk=2, hidden=16, dtype=0, y=P, ldy=16, stream=None)
COMBINE_GRAD = dict(dy=P, lddy=16, ys=P, ldys=16, rows=P, slots=P, weights=P, tokens=4, topk=2, hidden=16, dtype=0,
                    dys=P, lddys=16, dw=P, stream=None)


@pytest.mark.parametrize("name,base", [("gemm_moe_dispatch", DISPATCH), ("gemm_moe_dispatch_grad", DISPATCH_GRAD),
                                       ("gemm_moe_combine", COMBINE), ("gemm_moe_combine_grad", COMBINE_GRAD)])
def test_row_operator_refusals(name, base):
    fn = getattr(B, name)
    for key in base:
        if base[key] == P:
            refused(INV, fn, *_with(base, **{key: None}))
            refused(UNS, fn, *_with(base, **{key: P + 1}))
        if key.startswith("ld"):
            refused(INV, fn, *_with(base, **{key: 15}))
    for key in ("rows", "slots", "weights", "dw"):
        if key in base:
            refused(UNS, fn, *_with(base, **{key: P + 2}))
    for bad in (dict(tokens=-1), dict(topk=0), dict(hidden=-1), dict(dtype=2), dict(dtype=-1)):
        refused(INV, fn, *_with(base, **bad))
    refused(UNS, fn, *_with(base, tokens=2 ** 31))
    refused(UNS, fn, *_with(base, tokens=2 ** 62))
    refused(UNS, fn, *_with(base, topk=65536))
    refused(UNS, fn, *_with(base, **{"hidden": 2 ** 31, **{k: 2 ** 31 for k in base if k.startswith("ld")}}))
    fn(*_with(base, tokens=0))  # nothing to do, nothing launched


@pytest.mark.parametrize("status,args", [
    (INV, (2, 4, 8, 8, 8, 0, 0)), (INV, (0, 0, 8, 8, 8, 0, 0)), (INV, (0, 4, -1, 8, 8, 0, 0)),
    (INV, (0, 4, 8, -8, 8, 0, 0)), (INV, (0, 4, 8, 8, -8, 0, 0)), (INV, (0, 4, 8, 8, 8, 2, 0)),
    (INV, (0, 4, 8, 8, 8, 0, 2)), (UNS, (0, 1025, 8, 8, 8, 0, 0)), (UNS, (0, 4, 2 ** 31, 8, 8, 0, 0)),
    (UNS, (0, 4, 8, 12, 8, 0, 0)), (UNS, (1, 4, 8, 8, 20, 0, 0)), (UNS, (0, 4, 8, 2 ** 31, 8, 0, 0)),
    (UNS, (0, 4, 8, 8, 2 ** 31, 0, 0))])
def test_grouped_plan_refusals(status, args):
    refused(status, B.gemm_grouped_plan_create, *args)


def test_grouped_null_handles():
    lib = B.load()
    assert lib.gemm_grouped_plan_create(None, 0, 1, 8, 8, 8, 0, 0) == INV
    size = ctypes.c_size_t()
    assert lib.gemm_grouped_workspace_size(None, ctypes.byref(size)) == INV
    assert lib.gemm_grouped_run(None, P, P, P, P, P, None) == INV
    assert lib.gemm_grouped_last_status(None, None) == INV
    assert lib.gemm_grouped_plan_destroy(None) == B.GEMM_OK
