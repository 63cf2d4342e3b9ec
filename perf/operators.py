"""Cases that measure the 8-bit expert path: the residual RMS norm with an
8-bit output, the routing with groups, the block-scaled 8-bit product and the
experts of one layer in 8 bits.

Values in 8 bits are e4m3 with one float32 scale for each 128 consecutive
columns of a row (rows) or each 128 x 128 block (weights); a gate_up weight
(E, 2F, D) has the blocks of its gate half and of its up half apart:
(E, 2, ceil(F/128), ceil(D/128)).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
FP8_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one decode token between attention and the experts: a few rows, latency
        {"name": "norm decode", "op": "norm", "T": 4, "D": 4096, "dtype": "bf16", "residual": True, "quant": True},
        # the fine-grained layer's prefill, straight to 8 bits
        {"name": "norm prefill", "op": "norm", "T": 16384, "D": 2048, "dtype": "bf16", "residual": True, "quant": True},
        # a float32 stream of odd width without a residual (the first layer), norm only
        {"name": "norm f32 odd", "op": "norm", "T": 4099, "D": 2567, "dtype": "f32", "residual": False, "quant": False},
        # routing of one decode step: 256 experts in 8 groups
        {"name": "select decode", "op": "select", "T": 8, "E": 256, "K": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_score": "top2", "norm": True, "scale": 2.5, "masked": False},
        # the same router over a long prefill
        {"name": "select prefill", "op": "select", "T": 16384, "E": 256, "K": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_score": "top2", "norm": True, "scale": 2.5, "masked": False},
        # the fine-grained layer's router: softmax over 64 experts, some of them switched off, groups by their best expert
        {"name": "select softmax", "op": "select", "T": 5003, "E": 64, "K": 6, "score": "softmax", "bias": False,
         "groups": 8, "top_groups": 3, "group_score": "max", "norm": False, "scale": 1.0, "masked": True},
        # a dense projection for a few decode tokens: the weight stream
        {"name": "product 16 rows", "op": "product", "E": 1, "M": 16, "N": 4096, "K": 14336, "skew": 0.0},
        # a ragged batch over the fine-grained layer's 64 experts, some of them empty
        {"name": "product ragged", "op": "product", "E": 64, "M": 9973, "N": 1408, "K": 2048, "skew": 1.0},
        # one large dense product
        {"name": "product large", "op": "product", "E": 1, "M": 8192, "N": 4096, "K": 14336, "skew": 0.0},
        # one token through the experts of the decode layer
        {"name": "experts 1 token", "op": "experts", "T": 1, "D": 4096, "F": 14336, "E": 8, "K": 2, "skew": 0.0},
        # a decode step over 64 fine-grained experts
        {"name": "experts decode", "op": "experts", "T": 32, "D": 2048, "F": 1408, "E": 64, "K": 6, "skew": 0.5},
        # the prefill of the eight-expert layer
        {"name": "experts prefill", "op": "experts", "T": 4096, "D": 4096, "F": 14336, "E": 8, "K": 2, "skew": 0.2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "select", "product", "experts"])
    if op == "norm":
        T, D = _log(rng, 1, 16384), _log(rng, 64, 16384)
        D = min(D, max(64, (1 << 25) // T))
        if rng.random() < 0.7:
            D = (D + 7) // 8 * 8
        return {"op": op, "T": T, "D": D, "dtype": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.7,
                "quant": rng.random() < 0.7}
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 5, 8])
        size = rng.randint(max(2, -(-8 // groups)), 256 // groups)
        top = rng.randint(1, groups)
        return {"op": op, "T": _log(rng, 1, 16384), "E": groups * size, "K": rng.randint(1, min(8, top * size)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.6, "groups": groups,
                "top_groups": top, "group_score": rng.choice(["max", "top2"]), "norm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.random() < 0.3}
    if op == "product":
        E = rng.choice([1, 1, 4, 8, 16, 64])
        N, K = 8 * _log(rng, 16, 1024), 16 * _log(rng, 8, 896)
        M = _log(rng, 1, 8192)
        while 2 * E * N * K > (3 << 29) and E > 1:
            E //= 2
        return {"op": op, "E": E, "M": min(M, (8192 * 4096 * 14336) // (N * K)), "N": N, "K": K,
                "skew": round(rng.uniform(0, 1.5), 2)}
    E = rng.choice([4, 8, 16, 32, 64])
    D, F = 16 * _log(rng, 16, 256), 16 * _log(rng, 8, 896)
    while E > 4 and E * D * F > 8 * 4096 * 14336:
        E //= 2
    K = rng.randint(1, min(8, E))
    return {"op": op, "T": min(_log(rng, 1, 8192), 4096 * 4096 * 14336 * 2 // (D * F * K)), "D": D, "F": F, "E": E,
            "K": K, "skew": round(rng.uniform(0, 1.0), 2)}


def _weight(g, E, N, K, std):
    """Weights as a block quantiser leaves them: the largest of a block near the type's largest value."""
    q = torch.empty(E, N, K, dtype=E4M3, device="cuda")
    for e in range(E):
        w = torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16)
        q[e] = (w * 100.0).clamp_(-FP8_MAX, FP8_MAX).to(E4M3)
    s = torch.rand(E, -(-N // BLOCK), -(-K // BLOCK), generator=g, device="cuda")
    return q, (s * 0.4 + 0.8) * (std / 100.0)


def _rows(g, M, K):
    """Activations: each row's blocks quantised by their own largest value."""
    kb = -(-K // BLOCK)
    q = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    q = (q * 150.0).clamp_(-FP8_MAX, FP8_MAX).to(E4M3)
    return q, torch.exp(torch.randn(M, kb, generator=g, device="cuda") * 0.3) / 150.0


def _popularity(g, E, skew):
    """Expert popularity (rank + 1)^-skew in a shuffled order."""
    p = torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** -skew
    return p[torch.randperm(E, generator=g, device="cuda")]


def _plan(s, rows):
    """What a plain batched product needs to know of the row counts: experts with rows, and the most rows of one."""
    rows = rows.tolist()
    s["active"], s["most"] = max(1, sum(r > 0 for r in rows)), max(1, max(rows))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "norm":
        T, D = case["T"], case["D"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a residual stream of growing rows with a few large channels, the sublayer's output beside it
        s["x"] = torch.randn(T, D, generator=g, device="cuda").to(dt)
        s["weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        s["eps"] = 1e-6
        s["residual"] = s["sum"] = s["q"] = s["scales"] = None
        if case["residual"]:
            r = torch.randn(T, D, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
            r[:, torch.randperm(D, generator=g, device="cuda")[: max(1, D // 512)]] *= 20.0
            s["residual"] = r.to(dt)
            s["sum"] = torch.empty(T, D, dtype=dt, device="cuda")
        s["out"] = torch.empty(T, D, dtype=dt, device="cuda")
        if case["quant"]:
            s["q"] = torch.empty(T, D, dtype=E4M3, device="cuda")
            s["scales"] = torch.empty(T, -(-D // BLOCK), device="cuda")
        return s
    if op == "select":
        T, E = case["T"], case["E"]
        s["logits"] = torch.randn(T, E, generator=g, device="cuda") * 1.5
        if case["masked"]:
            off = torch.rand(E, generator=g, device="cuda") < 0.1
            s["logits"][:, off] = float("-inf")
        s["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        s["selected"] = torch.empty(T, case["K"], dtype=torch.int64, device="cuda")
        s["weights"] = torch.empty(T, case["K"], device="cuda")
        return s
    if op == "product":
        E, M, N, K = case["E"], case["M"], case["N"], case["K"]
        s["a"], s["a_scales"] = _rows(g, M, K)
        s["w"], s["w_scales"] = _weight(g, E, N, K, 0.02)
        s["out"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        s["offsets"] = None
        if E > 1:
            p = _popularity(g, E, case["skew"])
            p[torch.rand(E, generator=g, device="cuda") < 0.1] = 0.0
            p = p if float(p.sum()) > 0 else torch.ones_like(p)
            rows = torch.bincount(torch.multinomial(p, M, replacement=True, generator=g), minlength=E)
            s["offsets"] = torch.cat([rows.new_zeros(1), rows.cumsum(0)]).to(torch.int32)
            _plan(s, rows)
        return s
    T, D, F, E, K = (case[k] for k in ("T", "D", "F", "E", "K"))
    s["x"], s["x_scales"] = _rows(g, T, D)
    q, _ = _weight(g, E, 2 * F, D, 0.02)
    s["gate_up"] = q
    u = torch.rand(E, 2, -(-F // BLOCK), -(-D // BLOCK), generator=g, device="cuda")
    s["gate_up_scales"] = (u * 0.4 + 0.8) * 2e-4
    s["down"], s["down_scales"] = _weight(g, E, D, F, 0.02)
    p = _popularity(g, E, case["skew"]).log() - torch.empty(T, E, device="cuda").exponential_(generator=g).log()
    s["selected"] = p.topk(K, dim=1).indices
    w = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
    s["weights"] = w.sort(dim=1, descending=True).values.contiguous()
    s["out"] = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    _plan(s, torch.bincount(s["selected"].reshape(-1), minlength=E))
    return s


# ------------------------------------------------------------- the plain form
def _expand(s, rows, cols, by):
    """Scales of blocks of `by` rows by 128 columns, one for each element."""
    if by > 1:
        s = s.repeat_interleave(by, -2)[..., :rows, :]
    return s.repeat_interleave(BLOCK, -1)[..., :cols]


def _wide(q, s, by, to=torch.float32):
    """The values that q and its scales stand for."""
    return q.to(to) * _expand(s.to(to), q.shape[-2], q.shape[-1], by)


def _blocks(v):
    """(q, scales) of each row's blocks of 128; q rounded to e4m3, nearest even."""
    n = v.shape[-1]
    pad = torch.nn.functional.pad(v, (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))
    scale = pad.abs().amax(-1).clamp_min(SCALE_FLOOR) / FP8_MAX
    q = (pad / scale.unsqueeze(-1)).flatten(-2)[..., :n].clamp(-FP8_MAX, FP8_MAX)
    return q.to(E4M3), scale


def _norm(s, to):
    h = s["x"].to(to)
    if s["residual"] is not None:
        h = (h + s["residual"].to(to)).to(s["x"].dtype)
    h32 = h.to(to)
    y = h32 * torch.rsqrt(h32.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].to(to)
    out = [h] if s["residual"] is not None else []
    out.append(y.to(s["x"].dtype) if to == torch.float32 else y)
    return out + (list(_blocks(y)) if s["q"] is not None else [])


def _select(s):
    """Scores in 64 bits: which of two near scores is larger decides whole numbers."""
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    l = s["logits"].double()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = e.sum(1, keepdim=True)
        score = e / torch.where(total > 0, total, torch.ones_like(total))
    choice = l if s["bias"] is None else score + s["bias"].double()
    order = choice.sort(dim=1, descending=True, stable=True).indices
    if G > 1:
        by = choice if s["bias"] is not None or c["group_score"] == "max" else score
        per = by.view(T, G, E // G).sort(dim=2, descending=True).values
        per = per[:, :, 0] if c["group_score"] == "max" else per[:, :, :2].sum(2)
        kept = per.sort(dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.int8, device=l.device).scatter_(1, kept, 1)
        ranked = keep.gather(1, order // (E // G))
        order = order.gather(1, ranked.sort(dim=1, descending=True, stable=True).indices)
    sel = order[:, :K].contiguous()
    w = score.gather(1, sel)
    if c["norm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-9)
    return sel, w * c["scale"]


def _by_expert(s, starts, counts):
    """Rows of each expert that has any, padded to the most rows of one: experts (A,), rows (A, most), and whether each is one."""
    act = (counts == 0).to(torch.int8).sort(stable=True).indices[: s["active"]]
    i = torch.arange(s["most"], device=counts.device)
    live = i < counts[act].unsqueeze(1)
    return act, torch.where(live, starts[act].unsqueeze(1) + i, torch.zeros_like(live, dtype=starts.dtype)), live


def _product(s, to):
    a = _wide(s["a"], s["a_scales"], 1, to)
    if s["offsets"] is None:
        return a @ _wide(s["w"][0], s["w_scales"][0], BLOCK, to).T
    o = s["offsets"].long()
    act, rows, live = _by_expert(s, o[:-1], o[1:] - o[:-1])
    c = torch.bmm(a[rows], _wide(s["w"][act], s["w_scales"][act], BLOCK, to).transpose(1, 2))
    out = torch.empty(s["case"]["M"], s["case"]["N"], dtype=to, device="cuda")
    out[rows[live]] = c[live]
    return out


def _experts(s, to):
    c = s["case"]
    T, D, F, E, K = (c[k] for k in ("T", "D", "F", "E", "K"))
    flat = s["selected"].reshape(-1)
    order = flat.sort(stable=True).indices
    counts = torch.zeros(E, dtype=torch.int64, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    act, rows, live = _by_expert(s, counts.cumsum(0) - counts, counts)
    slot = order[rows]
    x = _wide(s["x"], s["x_scales"], 1, to)[slot // K]
    gate_up = s["gate_up"][act].unflatten(1, (2, F))
    gu = torch.bmm(x, _wide(gate_up, s["gate_up_scales"][act], BLOCK, to).flatten(1, 2).transpose(1, 2))
    gate, up = gu[..., :F], gu[..., F:]
    h = _wide(*_blocks(gate / (1.0 + torch.exp(-gate)) * up), 1, to)
    y = torch.bmm(h, _wide(s["down"][act], s["down_scales"][act], BLOCK, to).transpose(1, 2))
    each = torch.empty(T * K, D, dtype=to, device=flat.device)
    each[slot[live]] = y[live]
    return (each.view(T, K, D) * s["weights"].to(to).unsqueeze(2)).sum(1)


def run(state):
    s = state
    c = s["case"]
    if own:
        from mixture_experts_ffn_09_b200 import moe
        if c["op"] == "norm":
            moe.add_rmsnorm(s["x"], s["weight"], s["eps"], residual=s["residual"], sum_out=s["sum"], out=s["out"],
                            out8=s["q"], scales=s["scales"])
            return [t for t in (s["sum"], s["out"], s["q"], s["scales"]) if t is not None]
        if c["op"] == "select":
            moe.select_experts(s["logits"], c["K"], c["norm"], s["selected"], s["weights"], score=c["score"],
                               selection_bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                               group_score=c["group_score"], scale=c["scale"])
            return [s["selected"], s["weights"]]
        if c["op"] == "product":
            moe.gemm_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["out"], offsets=s["offsets"])
            return [s["out"]]
        if "workspace" not in s:      # kept by the program from its first call on
            n = moe.experts_workspace_size_fp8(c["T"], c["D"], c["F"], c["E"], c["K"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        moe.experts_forward_fp8(s["x"], s["x_scales"], s["selected"], s["weights"], s["gate_up"], s["gate_up_scales"],
                                s["down"], s["down_scales"], s["out"], workspace=s["workspace"])
        return [s["out"]]
    if c["op"] == "norm":
        return _norm(s, torch.float32)
    if c["op"] == "select":
        sel, w = _select(s)
        return [sel, w.float()]
    return [(_product if c["op"] == "product" else _experts)(s, torch.float32).bfloat16()]


# ------------------------------------------------------------------- the work
def work(case):
    c = case
    if c["op"] == "norm":
        T, D, e = c["T"], c["D"], 2 if c["dtype"] == "bf16" else 4
        b = T * D * e * (2 + 2 * c["residual"]) + D * e
        return {"bytes": b + (T * D + 4 * T * -(-D // BLOCK) if c["quant"] else 0), "flops": 8 * T * D}
    if c["op"] == "select":
        T, E, K = c["T"], c["E"], c["K"]
        return {"bytes": 4 * T * E + 12 * T * K + (4 * E if c["bias"] else 0), "flops": 8 * T * E}
    if c["op"] == "product":
        E, M, N, K = c["E"], c["M"], c["N"], c["K"]
        touched = E if E == 1 else 0.9 * E * (1.0 - (1.0 - 1.0 / E) ** M)
        return {"bytes": M * K + touched * N * K + 2 * M * N + 4 * M * -(-K // BLOCK), "flops": 2 * M * N * K}
    T, D, F, E, K = (c[k] for k in ("T", "D", "F", "E", "K"))
    touched = E * (1.0 - (1.0 - K / E) ** T)
    return {"bytes": T * D + 4 * T * -(-D // BLOCK) + touched * 3 * D * F + 2 * T * D + 12 * T * K,
            "flops": 6 * T * K * D * F}


# ----------------------------------------------------- from the definitions
def _exact_rows(q, s):
    """q times its block's scale, in 64 bits, one block of columns at a time."""
    v = q.double()
    for b in range(s.shape[1]):
        v[:, b * BLOCK:(b + 1) * BLOCK] *= s[:, b:b + 1].double()
    return v


def _exact_weight(q, s):
    v = q.double()
    for i in range(s.shape[0]):
        v[i * BLOCK:(i + 1) * BLOCK] *= s[i].double().repeat_interleave(BLOCK)[: v.shape[1]]
    return v


def _exact_blocks(v):
    q, s = torch.empty_like(v), []
    for b in range(0, v.shape[1], BLOCK):
        part = v[:, b:b + BLOCK]
        scale = torch.clamp(part.abs().max(1).values, min=SCALE_FLOOR) / FP8_MAX
        # to e4m3: three fraction bits at the value's exponent, never below the subnormals' step 2^-9
        t = part / scale[:, None]
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(t.abs().clamp_min(1e-30))), min=-6.0) - 3.0)
        q[:, b:b + BLOCK] = torch.clamp(torch.round(t / step) * step, -FP8_MAX, FP8_MAX)
        s.append(scale)
    return q, torch.stack(s, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        x = s["x"].double()
        outs = []
        if s["residual"] is not None:
            x = (x + s["residual"].double()).to(s["x"].dtype).double()
            outs.append(x)
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / c["D"] + s["eps"]) * s["weight"].double()
        outs.append(y)
        return outs + (list(_exact_blocks(y)) if c["quant"] else [])
    if c["op"] == "select":
        return _exact_select(s)
    if c["op"] == "product":
        a = _exact_rows(s["a"], s["a_scales"])
        ends = [0, c["M"]] if s["offsets"] is None else s["offsets"].tolist()
        out = torch.zeros(c["M"], c["N"], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            if ends[e + 1] > ends[e]:
                out[ends[e]:ends[e + 1]] = a[ends[e]:ends[e + 1]] @ _exact_weight(s["w"][e], s["w_scales"][e]).T
        return [out]
    F = c["F"]
    x = _exact_rows(s["x"], s["x_scales"])
    out = torch.zeros(c["T"], c["D"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        t, k = torch.nonzero(s["selected"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        half = s["gate_up"][e].split(F)
        gate = x[t] @ _exact_weight(half[0], s["gate_up_scales"][e, 0]).T
        up = x[t] @ _exact_weight(half[1], s["gate_up_scales"][e, 1]).T
        q, sc = _exact_blocks(gate * torch.sigmoid(gate) * up)
        y = _exact_rows(q, sc) @ _exact_weight(s["down"][e], s["down_scales"][e]).T
        out.index_add_(0, t, y * s["weights"][t, k].double()[:, None])
    return [out]


def _exact_select(s):
    """On the host, expert by expert in the order (chosen group, rank, index)."""
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    l = s["logits"].cpu().numpy().astype(np.float64)
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            p = np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(l) / (1.0 + np.exp(l)))
        else:
            p = np.exp(l - np.where(np.isfinite(l), l, -1e300).max(1)[:, None])
            p = np.nan_to_num(p / np.where(np.isfinite(l).any(1), p.sum(1), 1.0)[:, None])
    rank = l if s["bias"] is None else p + s["bias"].cpu().numpy().astype(np.float64)
    outside = np.zeros((T, E), bool)
    if G > 1:
        by = rank if s["bias"] is not None or c["group_score"] == "max" else p
        by = np.sort(by.reshape(T, G, E // G), axis=2)
        best = by[:, :, -1] if c["group_score"] == "max" else by[:, :, -1] + by[:, :, -2]
        place = np.lexsort((np.broadcast_to(np.arange(G), (T, G)), -best), axis=1).argsort(1)
        outside = np.repeat(place >= c["top_groups"], E // G, axis=1)
    sel = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -rank, outside), axis=1)[:, :K]
    w = np.take_along_axis(p, sel, 1)
    if c["norm"]:
        w = w / (w.sum(1, keepdims=True) + 1e-9)
    return [np.ascontiguousarray(sel), w * c["scale"]]
