"""The 8-bit path's definitions in float64, for the tests: block format,
residual RMS norm, routing with groups, block-scaled products, experts."""
import torch

BLOCK = 128
FP8_MAX = 448.0
FLOOR = 2.0 ** -100
F8 = torch.float8_e4m3fn


def nblk(n):
    return -(-n // BLOCK)


def spread(scales, rows, cols, block_rows=1):
    """One scale per element."""
    s = scales.double()
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, -2)[..., :rows, :]
    return s.repeat_interleave(BLOCK, -1)[..., :cols]


def wide(q, scales, block_rows=1):
    return q.double() * spread(scales, q.shape[-2], q.shape[-1], block_rows)


def amax_blocks(v, block_rows=1):
    r, c = v.shape[-2:]
    p = torch.nn.functional.pad(v.abs(), (0, nblk(c) * BLOCK - c, 0, -r % block_rows))
    p = p.unflatten(-1, (nblk(c), BLOCK)).unflatten(-3, (-1, block_rows))
    return p.amax((-1, -3))


def quantize(v, block_rows=1):
    """(values read back, scales, half steps): v in e4m3 blocks, float64."""
    s = amax_blocks(v, block_rows).clamp_min(FLOOR) / FP8_MAX
    se = spread(s, v.shape[-2], v.shape[-1], block_rows)
    t = v / se
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(1e-300))).clamp_min(-6.0) - 3.0)
    return torch.round(t / step) * step * se, s, step / 2 * se


def add_rmsnorm(x, residual, weight, eps):
    """(h in x's type, y)."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    d = h.double()
    return h, d / torch.sqrt(d.square().mean(-1, keepdim=True) + eps) * weight.double()


def select(logits, K, norm, score="softmax", selection_bias=None, groups=1, top_groups=0,
           group_score="max", scale=1.0):
    top_groups = top_groups or groups
    l = logits.double()
    l = torch.where(l.isnan(), torch.full_like(l, float("-inf")), l)
    l = l.clamp_max(torch.finfo(torch.float32).max)
    T, E = l.shape
    if score == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.where(m == float("-inf"), torch.zeros_like(l), torch.exp(l - m))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        s = torch.sigmoid(l)
    c = l
    if selection_bias is not None:
        c = s + selection_bias.double()
        c = torch.where(c.isnan(), torch.full_like(c, float("-inf")), c)
    idx = torch.arange(E, device=l.device).expand(T, E)
    allowed = torch.ones(T, E, dtype=torch.bool, device=l.device)
    if groups > 1:
        n = E // groups
        by = c if selection_bias is not None or group_score == "max" else s
        v = by.view(T, groups, n).sort(-1, descending=True).values
        v = v[..., 0] if group_score == "max" or n == 1 else v[..., 0] + v[..., 1]
        order = v.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        allowed = torch.zeros(T, groups, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        allowed = allowed.repeat_interleave(n, 1)
    sel = torch.empty(T, K, dtype=torch.int64, device=l.device)
    left = allowed.clone()
    for k in range(K):
        best = torch.where(left, c, torch.full_like(c, float("-inf"))).amax(1, keepdim=True)
        pick = torch.where(left & (c == best), idx, torch.full_like(idx, E)).amin(1)
        sel[:, k] = pick
        left.scatter_(1, pick[:, None], False)
    w = s.gather(1, sel)
    if norm:
        w = w / (w.sum(1, keepdim=True) + 1e-9)
    return sel, w * scale


def product(a, a_scales, w, w_scales, offsets):
    """(C, sum |a||w|, rows covered)."""
    A, M = wide(a, a_scales), a.shape[0]
    W = wide(w, w_scales, BLOCK)
    C = torch.zeros(M, w.shape[-2], dtype=torch.float64, device=a.device)
    S, live = C.clone(), torch.zeros(M, dtype=torch.bool, device=a.device)
    for e in range(len(offsets) - 1):
        r = slice(offsets[e], offsets[e + 1])
        C[r], S[r], live[r] = A[r] @ W[e].T, A[r].abs() @ W[e].abs().T, True
    return C, S, live


def experts(x, x_scales, selected, weights, gate_up, gate_up_scales, down, down_scales):
    """(out, out with an unrounded intermediate, bound on the rounding of h)."""
    T, K = selected.shape
    E, D, F = down.shape
    X = wide(x, x_scales)
    out = torch.zeros(T, D, dtype=torch.float64, device=x.device)
    raw, bound = out.clone(), out.clone()
    gu = wide(gate_up.view(E, 2, F, D), gate_up_scales, BLOCK)
    W = wide(down, down_scales, BLOCK)
    for k in range(K):
        for e in selected[:, k].unique().tolist():
            if not 0 <= e < E:
                continue
            t = (selected[:, k] == e).nonzero()[:, 0]
            g, u = X[t] @ gu[e, 0].T, X[t] @ gu[e, 1].T
            h = g * torch.sigmoid(g) * u
            q, _, half = quantize(h)
            w = weights[t, k].double()[:, None]
            out[t] += w * (q @ W[e].T)
            raw[t] += w * (h @ W[e].T)
            bound[t] += w.abs() * (half @ W[e].abs().T)
    return out, raw, bound
