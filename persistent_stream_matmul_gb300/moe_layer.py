"""A mixture-of-experts layer on the library's operators, as a program would
call them: a router, the experts' two products around an activation, and the
gradients of the experts' part: to its input, to the choices' weights and to the
experts' matrices.  The router's own gradient is not here; it starts from that
of the weights.

    python -m persistent_stream_matmul_gb300.moe_layer          # train step and decode, timed

The router's product runs through a GEMM plan, the experts' through grouped
plans; sorting, dispatch and combine through the gemm_moe functions.  torch
holds the buffers and does what is no operator here: top-k of the router's
logits and the activation.  Nothing reads a group size back to the host.
"""
from __future__ import annotations

import argparse

import torch

from . import _binding as B

_DTYPES = {torch.float16: B.GEMM_F16, torch.bfloat16: B.GEMM_BF16}


def _check(name, t, shape, dtypes, device):
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype not in dtypes or t.device != device:
        have = "%s %s on %s" % (t.dtype, tuple(t.shape), t.device) if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError("%s: %s %s on %s needed, not %s" % (name, " or ".join(map(str, dtypes)), shape, device, have))


def _contiguous(name, t, shape, dtypes, device):
    _check(name, t, shape, dtypes, device)
    if not t.is_contiguous():
        raise ValueError("%s: a contiguous tensor needed" % name)


def _leading(name, t, shape, dtypes, device):
    """The leading dimension of a matrix whose rows are contiguous."""
    _check(name, t, shape, dtypes, device)
    rows, cols = shape
    if (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        raise ValueError("%s: contiguous rows needed, not strides %s" % (name, t.stride()))
    return t.stride(0) if rows > 1 else cols


class MoELayer:
    """``experts`` experts of ``up`` (hidden -> inner), ReLU, ``down`` (inner -> hidden); each
    token goes to ``topk`` of them.  Weights are in the layout of a linear layer: router
    (experts, hidden), up (experts, inner, hidden), down (experts, hidden, inner).  hidden, inner
    and experts are multiples of 8.  One instance serves one number of tokens, on the current
    stream of the device that holds the weights; its plans and workspaces are made once.  Operands
    of another shape, type or device are refused with a ValueError."""

    def __init__(self, tokens, topk, router, up, down):
        if not isinstance(up, torch.Tensor) or up.dim() != 3 or up.dtype not in _DTYPES or not up.is_cuda:
            raise ValueError("up: a 16-bit (experts, inner, hidden) tensor on the GPU needed")
        experts, inner, hidden = up.shape
        self.tokens, self.topk, self.experts = tokens, topk, experts
        self.hidden, self.inner = hidden, inner
        self.router, self.up, self.down = router, up, down
        self.dtype, self.code, dev = up.dtype, _DTYPES[up.dtype], up.device
        self.device, self.saved = dev, None
        for name, t, shape in (("router", router, (experts, hidden)), ("up", up, tuple(up.shape)),
                               ("down", down, (experts, hidden, inner))):
            _contiguous(name, t, shape, (self.dtype,), dev)
        self._stream()
        slots = tokens * topk
        rows, col, row = B.GEMM_GROUPED_ROWS, B.GEMM_COL_MAJOR, B.GEMM_ROW_MAJOR
        self.router_plan = B.Plan(tokens, experts, hidden, self.code, row, col, "auto")
        plan = lambda kind, n, k, layout: B.GroupedPlan(kind, experts, slots, n, k, self.code, layout)  # noqa: E731
        self.up_plan = plan(rows, inner, hidden, col)
        self.down_plan = plan(rows, hidden, inner, col)
        # the same matrices read the other way round, and the products of the row pairs
        self.up_back, self.down_back = plan(rows, hidden, inner, row), plan(rows, inner, hidden, row)
        self.up_grad = plan(B.GEMM_GROUPED_INNER, inner, hidden, col)
        self.down_grad = plan(B.GEMM_GROUPED_INNER, hidden, inner, col)
        grouped = (self.up_plan, self.down_plan, self.up_back, self.down_back, self.up_grad, self.down_grad)
        size = max([p.workspace_size for p in grouped] + [B.gemm_moe_sort_workspace_size(tokens, topk, experts), 16])
        # one workspace for all but the router's plan, which keeps flags in its own
        # between runs: the calls follow one another on one stream
        self.workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        self.router_workspace = torch.empty(max(16, self.router_plan.workspace_size), dtype=torch.uint8, device=dev)
        self.plans = (self.router_plan, *grouped)

    def _new(self, *shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=self.up.device)

    def _stream(self):
        if torch.cuda.current_device() != self.device.index:
            raise ValueError("the current device is not the layer's, %s" % self.device)
        return torch.cuda.current_stream()

    def route(self, x):
        """(choices, weights) of every token: top-k of the router's logits, which the product
        rounds to the layer's type, and their softmax."""
        stream = self._stream()
        _check("x", x, (self.tokens, self.hidden), (self.dtype,), self.device)
        logits = self._new(self.tokens, self.experts)
        self.router_plan.run(x.contiguous(), self.router, logits, self.router_workspace, stream)
        top, ids = torch.topk(logits.float(), self.topk, dim=1)
        return ids, torch.softmax(top, dim=1)

    def forward(self, x, ids, weights):
        """y for x (tokens, hidden), choices (int32 or int64, of any row stride, as x; outside the
        experts: dropped) and fp32 weights; what the gradient needs is kept in ``self.saved``."""
        T, k, E, H, stream = self.tokens, self.topk, self.experts, self.hidden, self._stream()
        ldx = _leading("x", x, (T, H), (self.dtype,), self.device)
        ld_ids = _leading("ids", ids, (T, k), (torch.int64, torch.int32), self.device)
        _contiguous("weights", weights, (T, k), (torch.float32,), self.device)
        index = B.GEMM_INDEX_I64 if ids.dtype == torch.int64 else B.GEMM_INDEX_I32
        offsets, rows, slots = (self._new(n, dtype=torch.int32) for n in (E + 1, T * k, T * k))
        B.gemm_moe_sort(ids, index, ld_ids, T, k, E, offsets, rows, slots, self.workspace, stream)
        xs = self._new(T * k, H)
        B.gemm_moe_dispatch(x, ldx, rows, slots, T, k, H, self.code, xs, H, stream)
        a = self._new(T * k, self.inner)
        self.up_plan.run(xs, self.up, a, offsets, self.workspace, stream)
        a.relu_()
        ys = self._new(T * k, H)
        self.down_plan.run(a, self.down, ys, offsets, self.workspace, stream)
        y = self._new(T, H)
        B.gemm_moe_combine(ys, H, rows, weights, T, k, H, self.code, y, H, stream)
        self.saved = (offsets, rows, slots, weights, xs, a, ys)
        return y

    def backward(self, dy):
        """(dx, dweights, dup, ddown) of the last forward."""
        if self.saved is None:
            raise RuntimeError("backward before forward")
        T, k, H, stream = self.tokens, self.topk, self.hidden, self._stream()
        lddy = _leading("dy", dy, (T, H), (self.dtype,), self.device)
        offsets, rows, slots, weights, xs, a, ys = self.saved
        dys, dweights = self._new(T * k, H), self._new(T, k, dtype=torch.float32)
        B.gemm_moe_combine_grad(dy, lddy, ys, H, rows, slots, weights, T, k, H, self.code, dys, H, dweights, stream)
        ddown = torch.empty_like(self.down)
        self.down_grad.run(a, dys, ddown, offsets, self.workspace, stream)
        da = self._new(T * k, self.inner)
        self.down_back.run(dys, self.down, da, offsets, self.workspace, stream)
        da.masked_fill_(a <= 0, 0)
        dup = torch.empty_like(self.up)
        self.up_grad.run(xs, da, dup, offsets, self.workspace, stream)
        dxs = self._new(T * k, H)
        self.up_back.run(da, self.up, dxs, offsets, self.workspace, stream)
        dx = self._new(T, H)
        B.gemm_moe_dispatch_grad(dxs, H, rows, T, k, H, self.code, dx, H, stream)
        return dx, dweights, dup, ddown

    def check(self):
        """Raise if a device wait of any plan ran out since the last check."""
        stream = torch.cuda.current_stream()
        for p in self.plans:
            if p.last_status(stream) != B.GEMM_OK:
                raise B.GemmError(B.GEMM_ERR_TIMEOUT, "MoELayer")

    def close(self):
        for p in self.plans:
            p.close()


def _time(fn, steps):
    for _ in range(3):
        fn()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    begin.record()
    for _ in range(steps):
        fn()
    end.record()
    torch.cuda.synchronize()
    return begin.elapsed_time(end) / steps * 1e3


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)

    def weights(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

    router, up = weights(a.experts, a.hidden), weights(a.experts, a.inner, a.hidden)
    down = weights(a.experts, a.hidden, a.inner)
    for tokens in (a.tokens, 1):
        layer = MoELayer(tokens, a.topk, router, up, down)
        x = torch.randn(tokens, a.hidden, generator=g, device="cuda").bfloat16()
        ids, w = layer.route(x)
        y = layer.forward(x, ids, w)
        forward = _time(lambda: layer.forward(x, ids, w), a.steps)
        both = _time(lambda: (layer.forward(x, ids, w), layer.backward(y)), a.steps)
        layer.check()
        flops = 4.0 * tokens * a.topk * a.hidden * a.inner
        print("%6d tokens: forward %9.1f us (%.0f TFLOP/s), with gradients %9.1f us (%.0f TFLOP/s)"
              % (tokens, forward, flops / forward / 1e6, both, 3 * flops / both / 1e6))
        layer.close()


if __name__ == "__main__":
    main()
