"""Products in 8-bit floating point and what feeds them, case by case: inputs, one pass, its work and its exact values.

Three operators make the 8-bit form of a linear layer, with one fp32 scale for each 128 elements of the summed
dimension (a vector), or for each 128 x 128 of them (a block):

  quantize  a 16-bit matrix -> 8-bit values and their scales: vectors along the rows, along the columns, both of
            them in one pass, or blocks
  norm      root-mean-square norm of a row, after the residual's addition: 16-bit, or 8-bit with scales; its gradient
  scaled    C = A * B of 8-bit operands with scales, in any layout

``run`` computes them in a plain form from elementary torch operations (``own`` false)
or through the library's entry points (``own`` true).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
LEAST = 2.0 ** -100  # a group's scale is not below this over the type's largest value
GROUP = 128
EPS = 1e-5


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the activations of one generated token on their way into a product: nothing but latency
        {"name": "quantize_token", "op": "quantize", "kind": "rows", "rows": 1, "cols": 14336, "dtype": "bf16", "type": "e4m3"},
        # a weight matrix after an optimizer's step
        {"name": "quantize_weight", "op": "quantize", "kind": "blocks", "rows": 14336, "cols": 4096, "dtype": "bf16", "type": "e4m3"},
        # the gradient of a training batch of odd size, for both products of a backward pass
        {"name": "quantize_both_odd", "op": "quantize", "kind": "both", "rows": 5003, "cols": 2056, "dtype": "f16", "type": "e5m2"},
        # one generated token between two layers
        {"name": "norm_token", "op": "norm", "grad": False, "rows": 1, "hidden": 4096, "dtype": "bf16", "residual": True, "out": "q"},
        # a prefill: residual added, norm handed to an 8-bit product
        {"name": "norm_prefill", "op": "norm", "grad": False, "rows": 8192, "hidden": 4096, "dtype": "bf16", "residual": True, "out": "q"},
        # rows of odd length, 16-bit output
        {"name": "norm_odd", "op": "norm", "grad": False, "rows": 5003, "hidden": 2056, "dtype": "f16", "residual": False, "out": "y"},
        # training: gradient to the rows, with that of the residual stream, and to the weight
        {"name": "norm_grad_batch", "op": "norm", "grad": True, "rows": 16384, "hidden": 4096, "dtype": "bf16", "residual": True, "out": "y"},
        # one generated token through a projection: the matrix is read once
        {"name": "scaled_token", "op": "scaled", "M": 1, "N": 14336, "K": 4096, "a": "e4m3", "b": "e4m3", "out": "bf16",
         "layout_a": "row", "layout_b": "col", "scale_a": "vector", "scale_b": "block"},
        # a decoding batch through the projection back
        {"name": "scaled_decode", "op": "scaled", "M": 96, "N": 4096, "K": 14336, "a": "e4m3", "b": "e4m3", "out": "bf16",
         "layout_a": "row", "layout_b": "col", "scale_a": "vector", "scale_b": "block"},
        # a prefill: bound by the tensor cores
        {"name": "scaled_prefill", "op": "scaled", "M": 8192, "N": 14336, "K": 4096, "a": "e4m3", "b": "e4m3", "out": "bf16",
         "layout_a": "row", "layout_b": "col", "scale_a": "vector", "scale_b": "block"},
        # gradient to the rows, an odd number of them: the matrix read the other way round, gradients in e5m2
        {"name": "scaled_back_odd", "op": "scaled", "M": 4001, "N": 2048, "K": 1536, "a": "e5m2", "b": "e4m3", "out": "f16",
         "layout_a": "row", "layout_b": "row", "scale_a": "vector", "scale_b": "block"},
        # training: gradient to the matrix, summed over a batch, both operands with vectors along the tokens
        {"name": "scaled_wgrad", "op": "scaled", "M": 14336, "N": 4096, "K": 8192, "a": "e5m2", "b": "e4m3", "out": "f32",
         "layout_a": "col", "layout_b": "row", "scale_a": "vector", "scale_b": "vector"},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "norm", "scaled", "scaled"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "quantize":
        cols = _log(rng, 16, 1792) * 8 - (rng.randint(1, 7) if rng.random() < 0.2 else 0)
        # at most the elements of the largest listed one
        rows = _log(rng, 1, max(1, min(32768, int(5.8e7 / cols))))
        return {"op": op, "kind": rng.choice(("rows", "cols", "both", "blocks")), "rows": rows, "cols": cols,
                "dtype": dtype, "type": rng.choice(("e4m3", "e5m2"))}
    if op == "norm":
        hidden = _log(rng, 16, 2048) * 8 - (rng.randint(1, 7) if rng.random() < 0.2 else 0)
        grad = rng.random() < 0.4
        rows = _log(rng, 1, max(1, min(32768, int((6.7e7 if grad else 3.3e7) / hidden))))
        return {"op": op, "grad": grad, "rows": rows, "hidden": hidden, "dtype": dtype, "residual": rng.random() < 0.6,
                "out": rng.choice(("q", "q", "y", "both"))}
    kind = rng.choice(("forward", "forward", "back", "wgrad"))
    N, K = _log(rng, 8, 896) * 16, _log(rng, 8, 896) * 16
    # at most the products and the bytes of the largest listed one
    most = max(1, min(16384, int(4.8e11 / (N * K)), int(2.5e8 / (N + K))))
    M = _log(rng, 1, most)
    case = {"op": op, "M": M, "N": N, "K": K, "a": "e4m3", "b": "e4m3", "out": dtype, "layout_a": "row", "layout_b": "col",
            "scale_a": "vector", "scale_b": rng.choice(("block", "block", "vector"))}
    if kind == "back":
        case.update(a=rng.choice(("e5m2", "e4m3")), layout_b="row", scale_b="block")
    if kind == "wgrad":
        # the tokens are summed over, in any number; what M was is the matrix's other side
        case.update(M=N, N=K, K=M, a=rng.choice(("e5m2", "e4m3")), out=rng.choice(("f32", dtype)), layout_a="col", layout_b="row",
                    scale_b="vector")
    return case


# ---------------------------------------------------------------- plain quantisation
def _grouped(x, dim):
    """x with zeros up to a multiple of the group along `dim`, and that dimension cut in two."""
    n = x.shape[dim]
    padded = -(-n // GROUP) * GROUP
    if padded != n:
        shape = list(x.shape)
        shape[dim] = padded - n
        x = torch.cat([x, torch.zeros(shape, dtype=x.dtype, device=x.device)], dim)
    return x.unflatten(dim, (padded // GROUP, GROUP))


def _quantize(x, type, kind):
    """Values and scales of an fp32 matrix; `kind` says which elements share a scale."""
    rows, cols = x.shape
    if kind == "rows":
        g = _grouped(x, 1)                       # rows, groups, 128
        dims = (2,)
    elif kind == "cols":
        g = _grouped(x, 0)                       # groups, 128, cols
        dims = (1,)
    else:
        g = _grouped(_grouped(x, 0), 2)          # groups, 128, groups, 128
        dims = (1, 3)
    amax = g.abs().amax(dims, keepdim=True).clamp(min=LEAST)
    largest = torch.full_like(amax, LARGEST[type])
    # in 64 bits: between 16-bit values a quotient that lies on a border between two 8-bit ones is common
    q = (g.double() * largest.double() / amax.double()).float().reshape(g.shape[0] if kind == "rows" else g.shape[0] * GROUP, -1)
    scales = (amax / largest).squeeze(dims)
    if kind == "rows":
        scales = scales.t()
    return q[:rows, :cols].to(TYPES[type]), scales.contiguous()


def _spread(scales, rows, cols, kind):
    """The scale of every element of a stored matrix."""
    if kind == "rows":
        return scales.t().repeat_interleave(GROUP, 1)[:, :cols]
    if kind == "cols":
        return scales.repeat_interleave(GROUP, 0)[:rows]
    return scales.repeat_interleave(GROUP, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _activations(shape, g, dtype):
    """Rows of different size, as a network's activations have them."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.7 * torch.randn(shape[0], 1, generator=g, device="cuda"))
    return x.to(dtype)


def _kinds(case):
    """Which elements of the stored operands of a product share a scale."""
    a = "blocks" if case["scale_a"] == "block" else "rows" if case["layout_a"] == "row" else "cols"
    b = "blocks" if case["scale_b"] == "block" else "rows" if case["layout_b"] == "col" else "cols"
    return a, b


def _inputs(case, seed):
    g = _generator(seed)
    if case["op"] == "quantize":
        return {"x": _activations((case["rows"], case["cols"]), g, DTYPES[case["dtype"]])}
    if case["op"] == "norm":
        dt, shape = DTYPES[case["dtype"]], (case["rows"], case["hidden"])
        st = {"weight": (1.0 + 0.2 * torch.randn(shape[1], generator=g, device="cuda")).to(dt)}
        st["x"] = _activations(shape, g, dt)
        if case["grad"]:
            st["dy"] = _normal(shape, g, dt)
            st["rstd"] = torch.rsqrt(st["x"].float().square().mean(1) + EPS)
        if case["residual"]:
            st["residual"] = _normal(shape, g, dt, 2.0)
        return st
    M, N, K = case["M"], case["N"], case["K"]
    a = _activations((M, K) if case["layout_a"] == "row" else (K, M), g, torch.float32)
    b = _normal((N, K) if case["layout_b"] == "col" else (K, N), g, torch.float32, K ** -0.5)
    ka, kb = _kinds(case)
    st = {}
    st["a"], st["scales_a"] = _quantize(a, case["a"], ka)
    st["b"], st["scales_b"] = _quantize(b, case["b"], kb)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        _prepare_own(case, st)
    return st


def _prepare_own(case, st):
    import persistent_stream_matmul_gb300 as psm

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if case["op"] == "quantize":
        R, C, t = case["rows"], case["cols"], TYPES[case["type"]]
        r, c = -(-R // GROUP), -(-C // GROUP)
        out = {"rows": (empty(R, C, dtype=t), empty(c, R)), "cols": (empty(R, C, dtype=t), empty(r, C)),
               "blocks": (empty(R, C, dtype=t), empty(r, c))}
        st["out"] = out["rows"] + out["cols"] if case["kind"] == "both" else out[case["kind"]]
        return
    if case["op"] == "norm":
        R, H, dt = case["rows"], case["hidden"], DTYPES[case["dtype"]]
        if case["grad"]:
            st["out"] = (empty(R, H, dtype=dt), empty(H))
            st["workspace"] = empty(max(16, psm.gemm_rms_norm_grad_workspace_size(R, H)), dtype=torch.uint8)
            return
        st["sum"] = empty(R, H, dtype=dt) if case["residual"] else None
        st["y"] = empty(R, H, dtype=dt) if case["out"] != "q" else None
        st["q"] = empty(R, H, dtype=TYPES["e4m3"]) if case["out"] != "y" else None
        st["scales"] = empty(-(-H // GROUP), R) if case["out"] != "y" else None
        st["rstd"] = empty(R)
        st["out"] = tuple(st[n] for n in ("sum", "y", "q", "scales", "rstd") if st[n] is not None)
        return
    code = {"bf16": psm.GEMM_BF16, "f16": psm.GEMM_F16, "f32": psm.GEMM_F32, "e4m3": psm.GEMM_E4M3, "e5m2": psm.GEMM_E5M2,
            "row": psm.GEMM_ROW_MAJOR, "col": psm.GEMM_COL_MAJOR, "vector": psm.GEMM_SCALE_VECTOR, "block": psm.GEMM_SCALE_BLOCK}
    st["plan"] = psm.ScaledPlan(case["M"], case["N"], case["K"],
                                *(code[case[n]] for n in ("a", "b", "out", "layout_a", "layout_b", "scale_a", "scale_b")))
    st["workspace"] = empty(max(16, st["plan"].workspace_size), dtype=torch.uint8)
    st["out"] = empty(case["M"], case["N"], dtype=DTYPES[case["out"]])


# ---------------------------------------------------------------- one pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import persistent_stream_matmul_gb300 as psm
    case, out = st["case"], st["out"]
    stream = torch.cuda.current_stream()
    if case["op"] == "scaled":
        st["plan"].run(st["a"], st["scales_a"], st["b"], st["scales_b"], out, st["workspace"], stream)
        return out
    dtype = psm.GEMM_BF16 if case["dtype"] == "bf16" else psm.GEMM_F16
    if case["op"] == "quantize":
        R, C = case["rows"], case["cols"]
        type = psm.GEMM_E4M3 if case["type"] == "e4m3" else psm.GEMM_E5M2
        if case["kind"] == "both":
            psm.gemm_scaled_quantize_both(st["x"], C, R, C, dtype, type, out[0], C, out[1], out[2], C, out[3], stream)
        else:
            kind = {"rows": psm.GEMM_QUANTIZE_ROWS, "cols": psm.GEMM_QUANTIZE_COLS, "blocks": psm.GEMM_QUANTIZE_BLOCKS}[case["kind"]]
            psm.gemm_scaled_quantize(kind, st["x"], C, R, C, dtype, type, out[0], C, out[1], stream)
        return out
    R, H = case["rows"], case["hidden"]
    if case["grad"]:
        psm.gemm_rms_norm_grad(st["dy"], H, st["x"], H, st["weight"], st["rstd"], st.get("residual"), H, R, H, dtype,
                               out[0], H, out[1], st["workspace"], stream)
    else:
        psm.gemm_rms_norm(st["x"], H, st.get("residual"), H, st["weight"], EPS, R, H, dtype, st["sum"], H, st["y"], H,
                          st["q"], H, psm.GEMM_E4M3, st["scales"], st["rstd"], stream)
    return out


def _run_plain(st):
    case = st["case"]
    if case["op"] == "quantize":
        x = st["x"].float()
        if case["kind"] == "both":
            return _quantize(x, case["type"], "rows") + _quantize(x, case["type"], "cols")
        return _quantize(x, case["type"], case["kind"])
    if case["op"] == "norm":
        dt, w = DTYPES[case["dtype"]], st["weight"].float()
        if case["grad"]:
            s, dy, rstd = st["x"].float(), st["dy"].float(), st["rstd"][:, None]
            n = s * rstd
            wdy = w * dy
            dx = rstd * (wdy - n * (wdy * n).mean(1, keepdim=True))
            if case["residual"]:
                dx = dx + st["residual"].float()
            return dx.to(dt), (dy * n).sum(0, dtype=torch.float64).float()
        s, out = st["x"], ()
        if case["residual"]:
            s = (s.float() + st["residual"].float()).to(dt)
            out = (s,)
        s = s.float()
        rstd = torch.rsqrt(s.square().mean(1) + EPS)
        y = s * rstd[:, None] * w
        if case["out"] != "q":
            out += (y.to(dt),)
        if case["out"] != "y":
            out += _quantize(y, "e4m3", "rows")
        return out + (rstd,)
    ka, kb = _kinds(case)
    a = st["a"].float() * _spread(st["scales_a"], *st["a"].shape, ka)
    b = st["b"].float() * _spread(st["scales_b"], *st["b"].shape, kb)
    return torch.matmul(a if case["layout_a"] == "row" else a.t(), b if case["layout_b"] == "row" else b.t()).to(DTYPES[case["out"]])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "quantize":
        R, C = case["rows"], case["cols"]
        r, c = -(-R // GROUP), -(-C // GROUP)
        scales = {"rows": R * c, "cols": r * C, "blocks": r * c, "both": R * c + r * C}[case["kind"]]
        return {"bytes": R * C * (4 if case["kind"] == "both" else 3) + 4 * scales, "flops": 3 * R * C}
    if case["op"] == "norm":
        R, H = case["rows"], case["hidden"]
        if case["grad"]:
            return {"bytes": R * H * (8 if case["residual"] else 6) + 6 * H + 4 * R, "flops": 11 * R * H}
        size = (6 if case["residual"] else 2) + (2 if case["out"] != "q" else 0) + (1 if case["out"] != "y" else 0)
        return {"bytes": R * H * size + (4 * R * -(-H // GROUP) if case["out"] != "y" else 0) + 2 * H + 4 * R, "flops": 7 * R * H}
    M, N, K = case["M"], case["N"], case["K"]
    k = -(-K // GROUP)
    scales = k * (M if case["scale_a"] == "vector" else -(-M // GROUP)) + k * (N if case["scale_b"] == "vector" else -(-N // GROUP))
    return {"bytes": M * K + N * K + M * N * (4 if case["out"] == "f32" else 2) + 4 * scales, "flops": 2.0 * M * N * K}


# ---------------------------------------------------------------- exact values
def _to_grid(v, type):
    """The nearest values that the 8-bit type holds, ties to an even last digit."""
    digits, least = (3, -6) if type == "e4m3" else (2, -14)
    exponent = (torch.frexp(v).exponent.long() - 1).clamp(min=least) - digits
    step = ((exponent + 1023) << 52).view(torch.float64)  # 2 to that power, exactly
    return torch.round(v / step) * step


def _exact_quantized(x, type, kind):
    """The 8-bit values of a 64-bit matrix and their scales."""
    R, C = x.shape
    r, c = -(-R // GROUP), -(-C // GROUP)
    big = torch.zeros(r * GROUP, c * GROUP, dtype=torch.float64, device=x.device)
    big[:R, :C] = x.abs()
    big = big.view(r, GROUP, c, GROUP)
    peak = {"rows": lambda: big.amax(3).reshape(-1, c)[:R], "cols": lambda: big.amax(1).reshape(r, -1)[:, :C],
            "blocks": lambda: big.amax(3).amax(1)}[kind]()
    peak = torch.maximum(peak, torch.tensor(LEAST, dtype=torch.float64, device=x.device))
    scale = peak / LARGEST[type]
    at_r = torch.arange(R, device=x.device) // (1 if kind == "rows" else GROUP)
    at_c = torch.arange(C, device=x.device) // (1 if kind == "cols" else GROUP)
    return _to_grid(x * LARGEST[type] / peak[at_r][:, at_c], type), scale.t().contiguous() if kind == "rows" else scale


def exact(case, seed):
    st = _inputs(case, seed)
    f8 = torch.float64
    if case["op"] == "quantize":
        x = st["x"].to(f8)
        kinds = ("rows", "cols") if case["kind"] == "both" else (case["kind"],)
        return tuple(v for k in kinds for v in _exact_quantized(x, case["type"], k))
    if case["op"] == "norm":
        w, H = st["weight"].to(f8), case["hidden"]
        if case["grad"]:
            dx = torch.empty(st["x"].shape, dtype=f8, device="cuda")
            dw = torch.zeros(H, dtype=f8, device="cuda")
            for part in torch.split(torch.arange(case["rows"], device="cuda"), 4096):
                s, dy, r = st["x"][part].to(f8), st["dy"][part].to(f8), st["rstd"][part].to(f8)
                dot = torch.einsum("ij,ij,j->i", dy, s, w)
                dx[part] = torch.einsum("i,j,ij->ij", r, w, dy) - torch.einsum("i,ij->ij", dot * r ** 3 / H, s)
                if case["residual"]:
                    dx[part] += st["residual"][part].to(f8)
                dw += torch.einsum("ij,ij,i->j", dy, s, r)
            return dx, dw
        out = []
        s = st["x"].to(f8)
        if case["residual"]:
            # the norm is that of the sum as it is kept, in 16 bits
            out.append(s + st["residual"].to(f8))
            s = out[0].to(DTYPES[case["dtype"]]).to(f8)
        rstd = (torch.einsum("ij,ij->i", s, s) / H + EPS) ** -0.5
        y = torch.einsum("ij,i,j->ij", s, rstd, w)
        if case["out"] != "q":
            out.append(y)
        if case["out"] != "y":
            out.extend(_exact_quantized(y, "e4m3", "rows"))
        return (*out, rstd)
    M, N, K = case["M"], case["N"], case["K"]
    ka, kb = _kinds(case)

    def values(q, scales, kind):
        R, C = q.shape
        table = scales.t() if kind == "rows" else scales
        at_r = torch.arange(R, device="cuda") // (1 if kind == "rows" else GROUP)
        at_c = torch.arange(C, device="cuda") // (1 if kind == "cols" else GROUP)
        return q.to(torch.float32).to(f8) * table.to(f8)[at_r][:, at_c]

    a, b = values(st["a"], st["scales_a"], ka), values(st["b"], st["scales_b"], kb)
    a = a if case["layout_a"] == "row" else a.t()
    b = b if case["layout_b"] == "row" else b.t()
    out = torch.empty(M, N, dtype=f8, device="cuda")
    for rows in torch.split(torch.arange(M, device="cuda"), 2048):
        out[rows] = torch.einsum("mk,kn->mn", a[rows], b)
    return out
