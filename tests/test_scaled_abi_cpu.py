"""Refusals of the 8-bit linear layer's entry points.  They come before any
device call, so they need no GPU; the operands are addresses that are never
read.  And the gradient formula of the norm against differences."""
import ctypes

import pytest
import torch

from persistent_stream_matmul_gb300 import _binding as B
from persistent_stream_matmul_gb300 import build

P = 0x1000  # an aligned address
INV, UNS, WS = B.GEMM_ERR_INVALID_ARG, B.GEMM_ERR_UNSUPPORTED, B.GEMM_ERR_WORKSPACE
NAN = float("nan")


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


QUANTIZE = dict(kind=0, x=P, ldx=16, rows=4, cols=16, dtype=1, type=0, q=P, ldq=16, scales=P, stream=None)
BOTH = dict(x=P, ldx=16, rows=4, cols=16, dtype=1, type=0, q_rows=P, ldq_rows=16, scales_rows=P, q_cols=P, ldq_cols=16,
            scales_cols=P, stream=None)


@pytest.mark.parametrize("fn,base", [("gemm_scaled_quantize", QUANTIZE), ("gemm_scaled_quantize_both", BOTH)])
def test_quantize_refusals(fn, base):
    fn = getattr(B, fn)
    for key in base:
        if base[key] == P:
            refused(INV, fn, *_with(base, **{key: None}))
        if key.startswith("ld"):
            refused(INV, fn, *_with(base, **{key: 15}))
        if key.startswith("scales"):
            refused(UNS, fn, *_with(base, **{key: P + 2}))
    for bad in (dict(rows=-1), dict(cols=-1), dict(dtype=2), dict(dtype=-1), dict(type=2), dict(type=-1)):
        refused(INV, fn, *_with(base, **bad))
    if "kind" in base:
        refused(INV, fn, *_with(base, kind=3))
        refused(INV, fn, *_with(base, kind=-1))
    refused(UNS, fn, *_with(base, x=P + 1))
    refused(UNS, fn, *_with(base, rows=2 ** 31))
    refused(UNS, fn, *_with(base, cols=2 ** 31, **{k: 2 ** 31 for k in base if k.startswith("ld")}))
    fn(*_with(base, rows=0))  # nothing to do, nothing launched
    fn(*_with(base, cols=0))


NORM = dict(x=P, ldx=16, residual=P, ldres=16, weight=P, eps=1e-5, rows=4, hidden=16, dtype=1, sum=P, ldsum=16, y=P, ldy=16,
            q=P, ldq=16, type=0, scales=P, rstd=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INV, dict(x=None)), (INV, dict(weight=None)), (INV, dict(y=None, q=None, scales=None)), (INV, dict(q=None)),
    (INV, dict(scales=None)), (INV, dict(residual=None)), (INV, dict(rows=-1)), (INV, dict(hidden=-1)), (INV, dict(eps=-1e-9)),
    (INV, dict(eps=NAN)), (INV, dict(ldx=15)), (INV, dict(ldres=15)), (INV, dict(ldsum=15)), (INV, dict(ldy=15)),
    (INV, dict(ldq=15)), (INV, dict(dtype=2)), (INV, dict(type=2)), (UNS, dict(rows=2 ** 31)),
    (UNS, dict(hidden=32769, ldx=32769, ldres=32769, ldsum=32769, ldy=32769, ldq=32769)), (UNS, dict(x=P + 1)),
    (UNS, dict(residual=P + 1)), (UNS, dict(weight=P + 1)), (UNS, dict(sum=P + 1)), (UNS, dict(y=P + 1)), (UNS, dict(scales=P + 2)),
    (UNS, dict(rstd=P + 2))])
def test_norm_refusals(status, changes):
    refused(status, B.gemm_rms_norm, *_with(NORM, **changes))


GRAD = dict(dy=P, lddy=16, s=P, lds=16, weight=P, rstd=P, dsum=P, lddsum=16, rows=4, hidden=16, dtype=1, dx=P, lddx=16,
            dweight=P, workspace=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INV, dict(dy=None)), (INV, dict(s=None)), (INV, dict(weight=None)), (INV, dict(rstd=None)), (INV, dict(dx=None)),
    (INV, dict(rows=-1)), (INV, dict(hidden=-1)), (INV, dict(lddy=15)), (INV, dict(lds=15)), (INV, dict(lddsum=15)),
    (INV, dict(lddx=15)), (INV, dict(dtype=2)), (UNS, dict(rows=2 ** 31)),
    (UNS, dict(hidden=32769, lddy=32769, lds=32769, lddsum=32769, lddx=32769)), (UNS, dict(dy=P + 1)), (UNS, dict(s=P + 1)),
    (UNS, dict(weight=P + 1)), (UNS, dict(rstd=P + 2)), (UNS, dict(dsum=P + 1)), (UNS, dict(dx=P + 1)), (UNS, dict(dweight=P + 2)),
    (WS, dict(workspace=None)), (WS, dict(workspace=P + 8))])
def test_norm_grad_refusals(status, changes):
    refused(status, B.gemm_rms_norm_grad, *_with(GRAD, **changes))


def test_norm_without_rows_or_elements():
    for changes in (dict(rows=0), dict(hidden=0)):
        B.gemm_rms_norm(*_with(NORM, **changes))
    B.gemm_rms_norm_grad(*_with(GRAD, hidden=0))
    B.gemm_rms_norm_grad(*_with(GRAD, rows=0, dweight=None, workspace=None))
    for bad in ((-1, 16), (4, -1)):
        refused(INV, B.gemm_rms_norm_grad_workspace_size, *bad)
    refused(UNS, B.gemm_rms_norm_grad_workspace_size, 4, 32769)
    refused(UNS, B.gemm_rms_norm_grad_workspace_size, 2 ** 31, 16)
    assert B.load().gemm_rms_norm_grad_workspace_size(4, 16, None) == INV
    assert B.gemm_rms_norm_grad_workspace_size(0, 16) == 0


PLAN = dict(M=64, N=64, K=64, type_a=0, type_b=0, out=1, layout_a=0, layout_b=1, scale_a=0, scale_b=1)


@pytest.mark.parametrize("status,changes", [
    *[(INV, {k: -1}) for k in PLAN], *[(INV, {k: 2}) for k in ("type_a", "type_b", "layout_a", "layout_b", "scale_a", "scale_b")],
    (INV, dict(out=3)), (UNS, dict(M=2 ** 31)), (UNS, dict(N=2 ** 31)), (UNS, dict(K=2 ** 31)), (UNS, dict(K=72)),
    (UNS, dict(M=72, layout_a=1)), (UNS, dict(N=72, layout_b=0)), (UNS, dict(K=8, layout_b=0))])
def test_plan_refusals(status, changes):
    refused(status, B.gemm_scaled_plan_create, *_with(PLAN, **changes))


@pytest.mark.parametrize("M,N,K,ctas,form", [(1, 4096, 4096, 1, 2), (16, 65536, 4096, 1, 2), (17, 14336, 4096, 1, 1), (32, 128, 128, 1, 2), (33, 4096, 8192, 1, 0), (300, 256, 512, 1, 2),
                                             (129, 4096, 2048, 1, 0), (8192, 8192, 512, 2, 0)])
def test_offline_plans(M, N, K, ctas, form):
    p = B.ScaledPlan(M, N, K, 0, 0, 1, 0, 1, 0, 1, offline_sms=152)
    assert (p.info("ctas"), p.info("form")) == (ctas, form)
    if form != B.GEMM_SCALED_FEW:
        width = -(-M // 16) * 16 if form else 128 * ctas
        assert p.info("tile_width") == width and p.info("units") == 152 // ctas
        tiles = -(-N // 128) if form else -(-M // (128 * ctas)) * -(-N // (128 * ctas))
        assert p.info("tiles") == tiles
    assert (p.workspace_size > 0) == (p.info("shares") > 1)
    refused(B.GEMM_ERR_NO_DEVICE, p.run, P, P, P, P, P, P)
    assert p.last_status() == B.GEMM_ERR_NO_DEVICE
    for key, value, status in ((1, 3, UNS), (1, -1, UNS), (2, 3, UNS), (2, -2, UNS), (3, -2, UNS), (3, 0, B.GEMM_ERR_NO_DEVICE), (4, 0, INV)):
        refused(status, p.set_option, key, value)
    p.set_option(2, B.GEMM_SCALED_TURNED)
    p.set_option(1, 1)
    refused(UNS, p.set_option, 1, 2)  # a turned product has one CTA a unit
    assert p.info("ctas") == 1 and p.info("form") == B.GEMM_SCALED_TURNED
    refused(INV, p.info, 99)
    p.close()


def test_few_rows_need_contiguous_sums():
    for layouts in ((1, 1), (0, 0)):
        p = B.ScaledPlan(16, 64, 64, 0, 0, 1, *layouts, 0, 1, offline_sms=152)
        assert p.info("form") == B.GEMM_SCALED_TURNED
        refused(UNS, p.set_option, 2, B.GEMM_SCALED_FEW)


def test_offline_refusals():
    refused(INV, B.gemm_scaled_plan_create_offline, *PLAN.values(), 1)


def test_null_handles():
    lib = B.load()
    assert lib.gemm_scaled_plan_set_option(None, 1, 1) == INV
    assert lib.gemm_scaled_plan_get_info(None, 1, ctypes.byref(ctypes.c_int64())) == INV
    assert lib.gemm_scaled_plan_create(None, 16, 16, 16, 0, 0, 1, 0, 1, 0, 1) == INV
    assert lib.gemm_scaled_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == INV
    assert lib.gemm_scaled_run(None, P, P, P, P, P, P, None) == INV
    assert lib.gemm_scaled_last_status(None, None) == INV
    assert lib.gemm_scaled_plan_destroy(None) == B.GEMM_OK


def test_norm_gradient_formula_against_differences():
    """The formula that the kernels are held to, against central differences in 64 bits: their error
    is of order step^2 = 1e-10, and the function's values are below 10, so 1e-8 leaves two digits."""
    g = torch.Generator().manual_seed(3)
    R, H, eps, step = 3, 10, 1e-3, 1e-5
    s, dy = (torch.randn(R, H, generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.rand(H, generator=g, dtype=torch.float64) + 0.5

    def loss(s, w):
        return (dy * s * (s.square().mean(1, keepdim=True) + eps).rsqrt() * w).sum()

    rstd = (s.square().mean(1, keepdim=True) + eps).rsqrt()
    n = s * rstd
    ds = rstd * (w * dy - n * (w * dy * n).mean(1, keepdim=True))
    dw = (dy * n).sum(0)
    for i in range(R):
        for j in range(H):
            e = torch.zeros_like(s)
            e[i, j] = step
            assert abs((loss(s + e, w) - loss(s - e, w)) / (2 * step) - ds[i, j]) < 1e-8
    for j in range(H):
        e = torch.zeros_like(w)
        e[j] = step
        assert abs((loss(s, w + e) - loss(s, w - e)) / (2 * step) - dw[j]) < 1e-8
