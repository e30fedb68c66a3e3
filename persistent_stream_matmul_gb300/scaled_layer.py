"""A pre-norm feed-forward layer in 8-bit floating point on the library's
operators, as a program would call them: the residual's addition and the norm,
two linear layers around an activation, and the gradients to the input, the norm's
weight and both matrices.

    python -m persistent_stream_matmul_gb300.scaled_layer       # train step and decode, timed

Matrices are quantised in blocks of 128 x 128, rows in vectors of 128: along the
hidden dimension for the products forward and back, along the tokens for the
gradients of the matrices.  torch holds the buffers and computes the activation.
"""
from __future__ import annotations

import argparse

import torch

from . import _binding as B
from .moe_layer import _DTYPES, _check, _contiguous, _leading, _time

_FP8 = {B.GEMM_E4M3: torch.float8_e4m3fn, B.GEMM_E5M2: torch.float8_e5m2}


def _groups(n):
    return -(-n // B.GEMM_SCALE_GROUP)


class ScaledFeedForward:
    """``up`` (hidden -> inner), ReLU, ``down`` (inner -> hidden) behind a root-mean-square norm of
    x + residual.  Weights are in the layout of a linear layer and of one 16-bit type: norm
    (hidden), up (inner, hidden), down (hidden, inner); hidden and inner are multiples of 16.  They are
    quantised when the layer is made and by ``quantize_weights`` after they have changed.  One
    instance serves one number of tokens, on the current stream of the device that holds the
    weights; its plans and workspace are made once.  Gradients pass the products in
    ``grad_type``, e5m2 unless GEMM_E4M3 is asked for.  Operands of another shape, type or device are
    refused with a ValueError."""

    def __init__(self, tokens, norm, up, down, eps=1e-5, grad_type=B.GEMM_E5M2):
        if not isinstance(up, torch.Tensor) or up.dim() != 2 or up.dtype not in _DTYPES or not up.is_cuda:
            raise ValueError("up: a 16-bit (inner, hidden) tensor on the GPU needed")
        if grad_type not in _FP8:
            raise ValueError("grad_type: GEMM_E4M3 or GEMM_E5M2 needed")
        inner, hidden = up.shape
        self.tokens, self.hidden, self.inner, self.eps, self.grad_type = tokens, hidden, inner, eps, grad_type
        self.norm, self.up, self.down = norm, up, down
        self.dtype, self.code, self.device, self.saved = up.dtype, _DTYPES[up.dtype], up.device, None
        for name, t, shape in (("norm", norm, (hidden,)), ("up", up, (inner, hidden)), ("down", down, (hidden, inner))):
            _contiguous(name, t, shape, (self.dtype,), self.device)
        self._stream()
        e4, g, row, col = B.GEMM_E4M3, grad_type, B.GEMM_ROW_MAJOR, B.GEMM_COL_MAJOR
        vec, block, T = B.GEMM_SCALE_VECTOR, B.GEMM_SCALE_BLOCK, tokens
        plan = lambda M, N, K, ta, la, lb, sb: B.ScaledPlan(M, N, K, ta, e4, self.code, la, lb, vec, sb)  # noqa: E731
        self.up_plan, self.down_plan = plan(T, inner, hidden, e4, row, col, block), plan(T, hidden, inner, e4, row, col, block)
        # the same matrices read the other way round, and the sums over the tokens
        self.up_back, self.down_back = plan(T, hidden, inner, g, row, row, block), plan(T, inner, hidden, g, row, row, block)
        self.up_grad, self.down_grad = plan(inner, hidden, T, g, col, row, vec), plan(hidden, inner, T, g, col, row, vec)
        self.plans = (self.up_plan, self.down_plan, self.up_back, self.down_back, self.up_grad, self.down_grad)
        # one workspace: the calls follow one another on one stream
        size = max([p.workspace_size for p in self.plans] + [B.gemm_rms_norm_grad_workspace_size(T, hidden), 16])
        self.workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
        self.up8, self.down8 = (self._quantized(*w.shape, e4, (_groups(w.shape[0]), _groups(w.shape[1]))) for w in (up, down))
        self.quantize_weights()

    def _new(self, *shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)

    def _quantized(self, rows, cols, type, scales):
        return self._new(rows, cols, dtype=_FP8[type]), self._new(*scales, dtype=torch.float32)

    def _stream(self):
        if torch.cuda.current_device() != self.device.index:
            raise ValueError("the current device is not the layer's, %s" % self.device)
        return torch.cuda.current_stream()

    def quantize_weights(self):
        """Make the 8-bit forms of up and down again, after an optimizer's step."""
        stream = self._stream()
        for w, (q, s) in ((self.up, self.up8), (self.down, self.down8)):
            rows, cols = w.shape
            B.gemm_scaled_quantize(B.GEMM_QUANTIZE_BLOCKS, w, cols, rows, cols, self.code, B.GEMM_E4M3, q, cols, s, stream)

    def _along_rows(self, x, type, stream):
        rows, cols = x.shape
        q, s = self._quantized(rows, cols, type, (_groups(cols), rows))
        B.gemm_scaled_quantize(B.GEMM_QUANTIZE_ROWS, x, x.stride(0), rows, cols, self.code, type, q, cols, s, stream)
        return q, s

    def _along_tokens(self, x, type, stream):
        rows, cols = x.shape
        q, s = self._quantized(rows, cols, type, (_groups(rows), cols))
        B.gemm_scaled_quantize(B.GEMM_QUANTIZE_COLS, x, x.stride(0), rows, cols, self.code, type, q, cols, s, stream)
        return q, s

    def _both(self, x, ldx, type, stream):
        rows, cols = x.shape
        q, s = self._quantized(rows, cols, type, (_groups(cols), rows))
        qt, st = self._quantized(rows, cols, type, (_groups(rows), cols))
        B.gemm_scaled_quantize_both(x, ldx, rows, cols, self.code, type, q, cols, s, qt, cols, st, stream)
        return (q, s), (qt, st)

    def _run(self, plan, a, b, stream):
        out = self._new(plan.M, plan.N)
        plan.run(*a, *b, out, self.workspace, stream)
        return out

    def forward(self, x, residual, train=True):
        """(y, s): the layer's output and the residual stream s = x + residual, which the next layer adds
        y to.  x and residual: (tokens, hidden), of any row stride.  With ``train`` what the gradient
        needs is kept in ``self.saved``."""
        T, H, stream = self.tokens, self.hidden, self._stream()
        ldx = _leading("x", x, (T, H), (self.dtype,), self.device)
        ldr = _leading("residual", residual, (T, H), (self.dtype,), self.device)
        s, n = self._new(T, H), self._new(T, H) if train else None
        rstd = self._new(T, dtype=torch.float32) if train else None
        h8 = self._quantized(T, H, B.GEMM_E4M3, (_groups(H), T))
        B.gemm_rms_norm(x, ldx, residual, ldr, self.norm, self.eps, T, H, self.code, s, H, n, H, h8[0], H, B.GEMM_E4M3, h8[1], rstd, stream)
        a = self._run(self.up_plan, h8, self.up8, stream).relu_()
        y = self._run(self.down_plan, self._along_rows(a, B.GEMM_E4M3, stream), self.down8, stream)
        self.saved = (s, n, rstd, a) if train else None
        return y, s

    def backward(self, dy, ds=None):
        """(dx, dnorm, dup, ddown) of the last forward; dx is the gradient to x and to residual alike. ds:
        the gradient that reaches s past this layer.  dnorm is in fp32."""
        if self.saved is None:
            raise RuntimeError("backward without a forward for training")
        T, H, stream = self.tokens, self.hidden, self._stream()
        lddy = _leading("dy", dy, (T, H), (self.dtype,), self.device)
        ldds = 0 if ds is None else _leading("ds", ds, (T, H), (self.dtype,), self.device)
        s, n, rstd, a = self.saved
        g = self.grad_type
        dy8, dy8t = self._both(dy, lddy, g, stream)
        ddown = self._run(self.down_grad, dy8t, self._along_tokens(a, B.GEMM_E4M3, stream), stream)
        da = self._run(self.down_back, dy8, self.down8, stream).masked_fill_(a <= 0, 0)
        da8, da8t = self._both(da, self.inner, g, stream)
        dup = self._run(self.up_grad, da8t, self._along_tokens(n, B.GEMM_E4M3, stream), stream)
        dn = self._run(self.up_back, da8, self.up8, stream)
        dx, dnorm = self._new(T, H), self._new(H, dtype=torch.float32)
        B.gemm_rms_norm_grad(dn, H, s, H, self.norm, rstd, ds, ldds, T, H, self.code, dx, H, dnorm, self.workspace, stream)
        return dx, dnorm, dup, ddown

    def check(self):
        """Raise if a device wait of any plan ran out since the last check."""
        stream = torch.cuda.current_stream()
        for p in self.plans:
            if p.last_status(stream) != B.GEMM_OK:
                raise B.GemmError(B.GEMM_ERR_TIMEOUT, "ScaledFeedForward")

    def close(self):
        for p in self.plans:
            p.close()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()

    norm = torch.ones(a.hidden, device="cuda").bfloat16()
    up, down = normal(a.inner, a.hidden, scale=a.hidden ** -0.5), normal(a.hidden, a.inner, scale=a.inner ** -0.5)
    for tokens in (a.tokens, 1):
        layer = ScaledFeedForward(tokens, norm, up, down)
        x, r = normal(tokens, a.hidden), normal(tokens, a.hidden)
        y, s = layer.forward(x, r)
        forward = _time(lambda: layer.forward(x, r, train=False), a.steps)
        both = _time(lambda: (layer.forward(x, r), layer.backward(y, s)), a.steps)
        layer.check()
        flops = 4.0 * tokens * a.hidden * a.inner
        print("%6d tokens: forward %9.1f us (%.0f TFLOP/s), with gradients %9.1f us (%.0f TFLOP/s)"
              % (tokens, forward, flops / forward / 1e6, both, 3 * flops / both / 1e6))
        layer.close()


if __name__ == "__main__":
    main()
