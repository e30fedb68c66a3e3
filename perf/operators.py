"""The mixture-of-experts operators, case by case: their inputs, one pass, its work and its exact values.

Four operators make an expert layer around the library's products:

  sort      expert choices -> group offsets, the row of every (token, choice) slot, and back
  dispatch  token rows copied into expert order, or its gradient (summed back into tokens)
  combine   expert rows weighted and summed into tokens, or its gradient (rows and weights)
  grouped   one product per group of rows, or the gradient of the groups' matrices

``run`` computes them in a plain form from elementary torch operations (``own`` false)
or through the library's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # routing of one generated token: nothing but latency
        {"name": "sort_token", "op": "sort", "tokens": 1, "topk": 8, "experts": 64, "drop": 0.0, "skew": 0.0},
        # routing of a training batch over many small experts, 5 % of the slots dropped (padding)
        {"name": "sort_batch", "op": "sort", "tokens": 32768, "topk": 8, "experts": 256, "drop": 0.05, "skew": 1.0},
        # token rows of a prefill into expert order
        {"name": "dispatch_prefill", "op": "dispatch", "grad": False, "tokens": 8192, "topk": 2, "experts": 8,
         "hidden": 4096, "dtype": "bf16", "drop": 0.0, "skew": 0.0},
        # the gradient of that step in a training batch of odd size, some slots dropped
        {"name": "dispatch_grad_odd", "op": "dispatch", "grad": True, "tokens": 5003, "topk": 6, "experts": 64,
         "hidden": 2056, "dtype": "f16", "drop": 0.1, "skew": 1.0},
        # expert rows back into a decoding batch
        {"name": "combine_decode", "op": "combine", "grad": False, "tokens": 16, "topk": 8, "experts": 64,
         "hidden": 2048, "dtype": "f16", "drop": 0.0, "skew": 0.0},
        # training: gradients of the weighted sum, to the expert rows and to the router's weights
        {"name": "combine_grad_batch", "op": "combine", "grad": True, "tokens": 16384, "topk": 4, "experts": 32,
         "hidden": 4096, "dtype": "bf16", "drop": 0.0, "skew": 0.0},
        # one generated token through its 8 experts: eight single rows, eight matrices read once
        {"name": "grouped_token", "op": "grouped", "kind": "rows", "tokens": 1, "topk": 8, "experts": 64,
         "N": 1536, "K": 2048, "dtype": "bf16", "layout": "col", "drop": 0.0, "skew": 0.0},
        # a decoding batch through a few large experts: every matrix is read, two dozen rows each
        {"name": "grouped_decode", "op": "grouped", "kind": "rows", "tokens": 96, "topk": 2, "experts": 8,
         "N": 14336, "K": 4096, "dtype": "bf16", "layout": "col", "drop": 0.0, "skew": 0.0},
        # a prefill through the same experts: bound by the tensor cores
        {"name": "grouped_prefill", "op": "grouped", "kind": "rows", "tokens": 8192, "topk": 2, "experts": 8,
         "N": 14336, "K": 4096, "dtype": "bf16", "layout": "col", "drop": 0.0, "skew": 0.0},
        # gradient to the rows (the same matrices read the other way round), popular and idle experts
        {"name": "grouped_back_skewed", "op": "grouped", "kind": "rows", "tokens": 4001, "topk": 6, "experts": 64,
         "N": 2048, "K": 1536, "dtype": "f16", "layout": "row", "drop": 0.05, "skew": 1.0},
        # training: gradient of the large experts' matrices
        {"name": "grouped_wgrad", "op": "grouped", "kind": "inner", "tokens": 8192, "topk": 2, "experts": 8,
         "N": 14336, "K": 4096, "dtype": "bf16", "layout": "col", "drop": 0.0, "skew": 0.0},
        # gradient of many small matrices, popular and idle experts, some of them without a row
        {"name": "grouped_wgrad_skewed", "op": "grouped", "kind": "inner", "tokens": 509, "topk": 6, "experts": 128,
         "N": 1536, "K": 2048, "dtype": "f16", "layout": "row", "drop": 0.05, "skew": 1.5},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log8(rng, lo, hi):
    n = _log(rng, lo // 8, hi // 8) * 8
    return n + 8 if n == 3072 else n


def draw(rng):
    op = rng.choice(("sort", "dispatch", "combine", "grouped", "grouped"))
    experts = _log(rng, 1, 256)
    topk = rng.randint(1, min(8, experts))
    drop = rng.choice((0.0, 0.0, 0.05, 0.3))
    skew = rng.choice((0.0, 0.0, 0.7, 1.5))
    base = {"op": op, "topk": topk, "experts": experts, "drop": drop, "skew": skew}
    if op == "sort":
        return dict(base, tokens=_log(rng, 1, 32768))
    dtype = rng.choice(("bf16", "f16"))
    if op in ("dispatch", "combine"):
        hidden = _log8(rng, 256, 8192) - (rng.randint(1, 7) if rng.random() < 0.2 else 0)
        # at most the bytes of the largest listed gradient of the sum
        tokens = _log(rng, 1, max(1, min(32768, int(1.1e9 / (2 * hidden * (1 + 2 * topk))))))
        return dict(base, grad=rng.random() < 0.5, tokens=tokens, hidden=hidden, dtype=dtype)
    K = _log8(rng, 128, 8192)
    N = _log8(rng, 128, 14336)
    experts = base["experts"] = max(1, min(experts, int(1e9 / (2 * K * N))))
    topk = base["topk"] = min(topk, experts)
    # at most the products and the rows of the largest listed case
    tokens = _log(rng, 1, max(1, min(8192, int(1.7e12 / (2.0 * topk * K * N)), int(5e8 / (2.0 * topk * (K + N))))))
    return dict(base, kind=rng.choice(("rows", "rows", "inner")), tokens=tokens, N=N, K=K, dtype=dtype,
                layout=rng.choice(("col", "row")))


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _choices(case, g):
    """Expert choices of every token, distinct within a token; -1 where a slot is dropped."""
    T, k, E = case["tokens"], case["topk"], case["experts"]
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    logits = -torch.log(-torch.log(u)) - case["skew"] * torch.log(1.0 + torch.arange(E, device="cuda"))
    ids = torch.topk(logits, k, dim=1).indices
    if case["drop"] > 0:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["drop"], -1, ids)
    return ids.contiguous()


def _normal(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _inputs(case, seed):
    g = _generator(seed)
    ids = _choices(case, g)
    if case["op"] == "sort":
        return {"ids": ids}
    T, k = case["tokens"], case["topk"]
    offsets, rows, slots = _plain_sort(ids, case["experts"])
    st = {"rows": rows, "slots": slots, "offsets": offsets}
    dt = DTYPES[case["dtype"]]
    if case["op"] == "dispatch":
        st["x"] = _normal((T * k if case["grad"] else T, case["hidden"]), dt, g)
    elif case["op"] == "combine":
        st["ys"] = _normal((T * k, case["hidden"]), dt, g)
        st["weights"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), dim=1)
        if case["grad"]:
            st["dy"] = _normal((T, case["hidden"]), dt, g)
    else:
        E, K, N = case["experts"], case["K"], case["N"]
        st["a"] = _normal((T * k, K), dt, g)
        if case["kind"] == "rows":
            st["b"] = torch.empty((E, N, K) if case["layout"] == "col" else (E, K, N), dtype=dt, device="cuda")
            for e in range(E):
                st["b"][e] = _normal(st["b"].shape[1:], dt, g, K ** -0.5)
        else:
            st["b"] = _normal((T * k, N), dt, g)
        st["counts"] = (offsets[1:] - offsets[:-1]).tolist()  # a plain program loops over the groups
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        _prepare_own(case, st)
    return st


def _prepare_own(case, st):
    import persistent_stream_matmul_gb300 as psm
    T, k, E = case["tokens"], case["topk"], case["experts"]

    def empty(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if case["op"] == "sort":
        st["out"] = (empty(E + 1), empty(T, k), empty(T * k))
        st["workspace"] = empty(max(1, psm.gemm_moe_sort_workspace_size(T, k, E)), dtype=torch.uint8)
        return
    dt = DTYPES[case["dtype"]]
    if case["op"] == "dispatch":
        st["out"] = empty(T if case["grad"] else T * k, case["hidden"], dtype=dt)
    elif case["op"] == "combine":
        if case["grad"]:
            st["out"] = (empty(T * k, case["hidden"], dtype=dt), empty(T, k, dtype=torch.float32))
        else:
            st["out"] = empty(T, case["hidden"], dtype=dt)
    else:
        K, N = case["K"], case["N"]
        inner = case["kind"] == "inner"
        st["plan"] = psm.GroupedPlan(psm.GEMM_GROUPED_INNER if inner else psm.GEMM_GROUPED_ROWS, E, T * k, N, K,
                                     psm.GEMM_BF16 if case["dtype"] == "bf16" else psm.GEMM_F16,
                                     psm.GEMM_COL_MAJOR if case["layout"] == "col" else psm.GEMM_ROW_MAJOR)
        st["workspace"] = empty(max(1, st["plan"].workspace_size), dtype=torch.uint8)
        if inner:
            st["out"] = empty(*((E, N, K) if case["layout"] == "col" else (E, K, N)), dtype=dt)
        else:
            st["out"] = empty(T * k, N, dtype=dt)


# ---------------------------------------------------------------- one pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import persistent_stream_matmul_gb300 as psm
    case = st["case"]
    T, k = case["tokens"], case["topk"]
    stream = torch.cuda.current_stream()
    out = st["out"]
    if case["op"] == "sort":
        psm.gemm_moe_sort(st["ids"], psm.GEMM_INDEX_I64, k, T, k, case["experts"], *out, st["workspace"], stream)
        return out
    if case["op"] == "grouped":
        st["plan"].run(st["a"], st["b"], out, st["offsets"], st["workspace"], stream)
        return out
    H = case["hidden"]
    dtype = psm.GEMM_BF16 if case["dtype"] == "bf16" else psm.GEMM_F16
    if case["op"] == "dispatch" and case["grad"]:
        psm.gemm_moe_dispatch_grad(st["x"], H, st["rows"], T, k, H, dtype, out, H, stream)
    elif case["op"] == "dispatch":
        psm.gemm_moe_dispatch(st["x"], H, st["rows"], st["slots"], T, k, H, dtype, out, H, stream)
    elif case["grad"]:
        psm.gemm_moe_combine_grad(st["dy"], H, st["ys"], H, st["rows"], st["slots"], st["weights"], T, k, H, dtype,
                                  out[0], H, out[1], stream)
    else:
        psm.gemm_moe_combine(st["ys"], H, st["rows"], st["weights"], T, k, H, dtype, out, H, stream)
    return out


def _plain_sort(ids, E):
    """Offsets of the groups, the row of every slot and the slot of every row, in slot order within a group."""
    flat = ids.reshape(-1)
    n = flat.numel()
    ok = (flat >= 0) & (flat < E)
    key = torch.where(ok, flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(counts[:E], 0)
    at = torch.arange(n, device=ids.device)
    rows = torch.empty_like(key)
    rows[order] = at
    rows = torch.where(ok, rows, -1)
    slots = torch.where(at < offsets[E], order, -1)
    return offsets.int(), rows.int().reshape(ids.shape), slots.int()


def _run_plain(st):
    case = st["case"]
    k = case["topk"]
    if case["op"] == "sort":
        return _plain_sort(st["ids"], case["experts"])
    dt = DTYPES[case["dtype"]]
    rows, slots = st["rows"], st["slots"]
    if case["op"] == "dispatch":
        if case["grad"]:
            picked = st["x"][rows.clamp(min=0)].float()
            return torch.where((rows >= 0)[..., None], picked, 0.0).sum(1).to(dt)
        return torch.where((slots >= 0)[:, None], st["x"][slots.clamp(min=0) // k], 0.0)
    if case["op"] == "combine":
        w = st["weights"]
        if case["grad"]:
            dy = st["dy"].float()
            s = slots.clamp(min=0)
            dys = torch.where((slots >= 0)[:, None], dy[s // k] * w.reshape(-1)[s][:, None], 0.0).to(dt)
            dw = torch.where(rows >= 0, (st["ys"][rows.clamp(min=0)].float() * dy[:, None, :]).sum(2), 0.0)
            return dys, dw
        picked = st["ys"][rows.clamp(min=0)].float()
        return torch.where((rows >= 0)[..., None], picked * w[..., None], 0.0).sum(1).to(dt)
    a, b, col = st["a"], st["b"], case["layout"] == "col"
    at = 0
    if case["kind"] == "rows":
        out = torch.zeros((a.shape[0], case["N"]), dtype=dt, device="cuda")
        for e, n in enumerate(st["counts"]):
            if n:
                m = b[e].float()
                out[at:at + n] = torch.matmul(a[at:at + n].float(), m.t() if col else m).to(dt)
                at += n
        return out
    E, K, N = case["experts"], case["K"], case["N"]
    out = torch.zeros((E, N, K) if col else (E, K, N), dtype=dt, device="cuda")
    for e, n in enumerate(st["counts"]):
        if n:
            x, d = a[at:at + n].float(), b[at:at + n].float()
            out[e] = (torch.matmul(d.t(), x) if col else torch.matmul(x.t(), d)).to(dt)
            at += n
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def _active(case):
    """Expected number of experts that some token chose."""
    p = [(1.0 + e) ** -case["skew"] for e in range(case["experts"])]
    s = sum(p)
    keep = 1.0 - case["drop"]
    return sum(1.0 - (1.0 - min(1.0, case["topk"] * x / s) * keep) ** case["tokens"] for x in p)


def work(case):
    T, k, E = case["tokens"], case["topk"], case["experts"]
    slots = T * k
    kept = slots * (1.0 - case["drop"])
    if case["op"] == "sort":
        return {"bytes": 8 * slots + 4 * (E + 1) + 8 * slots, "flops": slots}
    if case["op"] == "dispatch":
        H = case["hidden"]
        if case["grad"]:
            return {"bytes": 2 * H * (kept + T) + 4 * slots, "flops": kept * H}
        return {"bytes": 2 * H * (T + slots) + 8 * slots, "flops": 0}
    if case["op"] == "combine":
        H = case["hidden"]
        if case["grad"]:
            return {"bytes": 2 * H * (T + kept + slots) + 16 * slots, "flops": 3 * kept * H}
        return {"bytes": 2 * H * (kept + T) + 8 * slots, "flops": 2 * kept * H}
    K, N = case["K"], case["N"]
    flops = 2.0 * kept * K * N
    if case["kind"] == "rows":
        return {"bytes": 2 * (kept * K + _active(case) * K * N + slots * N) + 4 * (E + 1), "flops": flops}
    return {"bytes": 2 * (kept * (K + N) + E * K * N) + 4 * (E + 1), "flops": flops}


# ---------------------------------------------------------------- exact values
def _members(st, E):
    """(expert, its slots in order, its first row), from the choices alone."""
    at = 0
    for e in range(E):
        mine = np.flatnonzero(st == e)
        yield e, mine, at
        at += len(mine)


def exact(case, seed):
    st = _inputs(case, seed)
    T, k, E = case["tokens"], case["topk"], case["experts"]
    ids = _choices(case, _generator(seed)).reshape(-1).cpu().numpy()
    f8 = torch.float64
    if case["op"] == "sort":
        offsets = np.zeros(E + 1, dtype=np.int64)
        rows, slots = np.full(T * k, -1, dtype=np.int64), np.full(T * k, -1, dtype=np.int64)
        for e, mine, at in _members(ids, E):
            offsets[e + 1] = at + len(mine)
            rows[mine] = at + np.arange(len(mine))
            slots[at:at + len(mine)] = mine
        return torch.from_numpy(offsets), torch.from_numpy(rows.reshape(T, k)), torch.from_numpy(slots)
    if case["op"] in ("dispatch", "combine"):
        H = case["hidden"]
        # (row, slot) of every slot that is kept
        pairs = [(at + np.arange(len(mine)), mine) for _, mine, at in _members(ids, E) if len(mine)]
        row = torch.from_numpy(np.concatenate([p[0] for p in pairs] or [np.zeros(0, int)])).cuda()
        slot = torch.from_numpy(np.concatenate([p[1] for p in pairs] or [np.zeros(0, int)])).cuda()
        token = torch.div(slot, k, rounding_mode="floor")
        if case["op"] == "dispatch" and not case["grad"]:
            out = torch.zeros((T * k, H), dtype=f8, device="cuda")
            out[row] = st["x"].to(f8)[token]
            return out
        scale = torch.ones(T * k, dtype=f8, device="cuda")
        if case["op"] == "combine":
            scale = st["weights"].reshape(-1).to(f8)
        if case["op"] == "dispatch" or not case["grad"]:
            out = torch.zeros((T, H), dtype=f8, device="cuda")
            src = st["x"] if case["op"] == "dispatch" else st["ys"]
            for j in range(k):
                here = (slot % k) == j
                out[token[here]] += src[row[here]].to(f8) * scale[slot[here]][:, None]
            return out
        dys = torch.zeros((T * k, H), dtype=f8, device="cuda")
        dw = torch.zeros(T * k, dtype=f8, device="cuda")
        for part in torch.split(torch.arange(len(row), device="cuda"), 16384):
            r, s, dy = row[part], slot[part], st["dy"][token[part]].to(f8)
            dys[r] = dy * scale[s][:, None]
            dw[s] = torch.einsum("ij,ij->i", dy, st["ys"][r].to(f8))
        return dys, dw.reshape(T, k)
    K, N, col = case["K"], case["N"], case["layout"] == "col"
    rows_kind = case["kind"] == "rows"
    out = torch.zeros((T * k, N) if rows_kind else ((E, N, K) if col else (E, K, N)), dtype=f8, device="cuda")
    for e, mine, at in _members(ids, E):
        if not len(mine):
            continue
        rng = slice(at, at + len(mine))
        a, b = st["a"][rng].to(f8), (st["b"][e] if rows_kind else st["b"][rng]).to(f8)
        if rows_kind:
            out[rng] = torch.einsum("rk,nk->rn" if col else "rk,kn->rn", a, b)
        else:
            out[e] = torch.einsum("rk,rn->nk" if col else "rk,rn->kn", a, b)
    return out
