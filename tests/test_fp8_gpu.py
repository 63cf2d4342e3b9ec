"""The 8-bit path on the GPU against float64 (tests/fp8_lib.py)."""
import threading

import pytest
import torch

import fp8_lib as R
from mixture_experts_ffn_09_b200 import moe

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
U32 = 2.0 ** -24                       # half a step of fp32
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def healthy():
    yield
    torch.cuda.synchronize()
    assert moe.device_status() == moe.MOE_OK


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, seed=0, std=1.0):
    return torch.randn(*shape, generator=gen(seed), device="cuda") * std


def rows8(M, K, seed):
    q = (randn(M, K, seed=seed) * 150).clamp(-448, 448).to(F8)
    return q, torch.exp(randn(M, R.nblk(K), seed=seed + 1) * 0.5) / 150


def weight8(E, N, K, seed, std=0.05):
    q = (randn(E, N, K, seed=seed) * 100).clamp(-448, 448).to(F8)
    return q, (torch.rand(E, R.nblk(N), R.nblk(K), generator=gen(seed + 1), device="cuda") + 0.5) * std / 100


# --------------------------------------------------------------------- norm
def run_norm(x, r, w, eps, sum_out=True, out=True, quant=True):
    T, D = x.shape
    o = dict(sum_out=torch.empty_like(x) if sum_out else None, out=torch.empty_like(x) if out else None,
             out8=torch.empty(T, D, dtype=F8, device="cuda") if quant else None,
             scales=torch.empty(T, R.nblk(D), device="cuda") if quant else None)
    moe.add_rmsnorm(x, w, eps, residual=r, **o)
    return o


def check_norm(x, r, w, eps, o):
    h, y = R.add_rmsnorm(x, r, w, eps)
    # mean of squares: at most 32 terms a lane, 10 levels of a tree, halved by the root;
    # root, quotient and two products: 2 steps each at most
    rel = (21 + 8) * U32
    if o["sum_out"] is not None:
        assert torch.equal(o["sum_out"], h)
    if o["out"] is not None:
        err = (o["out"].double() - y).abs()
        assert (err <= y.abs() * (rel + HALF[x.dtype] * (1 + rel)) + 1e-37).all()
    if o["out8"] is not None:
        _, s, half = R.quantize(y)
        assert ((o["scales"].double() - s).abs() <= s * (rel + 2 * U32)).all()
        # half a step of e4m3 (a value at the end of a binade may use the next one's step), and the scale's error
        err = (R.wide(o["out8"], o["scales"]) - y).abs()
        assert (err <= torch.maximum(half, y.abs() * 2.0 ** -4) * (1 + 1e-4) + y.abs() * (2 * rel + 8 * U32)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (1, 128), (5, 130), (33, 264), (2, 4096), (7, 2567),
                                 (1000, 96), (3, 8192), (2, 8200), (2, 16376), (3, 16384), (2, 32768),
                                 (2, 8193), (2, 16383), (2, 32761),
                                 (400, 5), (400, 130), (400, 259), (400, 516), (400, 1020), (400, 1032), (400, 2567),
                                 (300, 16383), (300, 32761), (300, 32768)])      # more rows than SMs take at once
def test_norm(dtype, T, D):
    x, r = randn(T, D, seed=1).to(dtype), randn(T, D, seed=2, std=3.0).to(dtype)
    w = (1 + 0.3 * randn(D, seed=3)).to(dtype)
    check_norm(x, r, w, 1e-6, run_norm(x, r, w, 1e-6))
    check_norm(x, None, w, 0.5, run_norm(x, None, w, 0.5, sum_out=T % 2 == 0))


@pytest.mark.parametrize("out,quant,sum_out", [(True, False, False), (False, True, True), (False, True, False)])
def test_norm_outputs(out, quant, sum_out):
    x, r, w = (randn(9, 520, seed=s).bfloat16() for s in (1, 2, 3))
    w = w[0].contiguous()
    check_norm(x, r, w, 1e-5, run_norm(x, r, w, 1e-5, sum_out, out, quant))


@pytest.mark.parametrize("D", [512, 515])
def test_norm_in_place_and_repeatable(D):
    x, r, w = randn(64, D, seed=1).bfloat16(), randn(64, D, seed=2).bfloat16(), randn(D, seed=3).bfloat16()
    want = run_norm(x, r, w, 1e-6)
    for _ in range(2):
        x2, r2 = x.clone(), r.clone()
        moe.add_rmsnorm(x2, w, 1e-6, residual=r2, sum_out=r2, out=x2)
        assert torch.equal(r2, want["sum_out"]) and torch.equal(x2, want["out"])


@pytest.mark.parametrize("D", [256, 259])
def test_norm_extremes(D):
    """Rows of zeros, of huge and tiny values, and non-finite ones that stay in their row."""
    x = randn(8, D, seed=4)
    x[0] = 0.0
    x[1] *= 1e18
    x[2] *= 1e-30
    x[3, :128] = 0.0                   # a block of zeros beside others
    x[4, 5] = NAN
    x[5, 5] = INF
    w = torch.ones(D, device="cuda")
    o = run_norm(x, None, w, 1e-6)
    fine = [0, 1, 2, 3, 6, 7]
    check_norm(x[fine], None, w, 1e-6, {k: v[fine] for k, v in o.items()})
    assert o["out"][4].isnan().all()
    assert o["out8"][4].float().isnan().all()
    assert o["out"][5].isnan().sum() == 1 and R.wide(o["out8"], o["scales"])[5, :128].isnan().any()
    assert (o["out8"][0].float() == 0).all() and (o["scales"] > 0).all()


# ----------------------------------------------------------------- quantise
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,block_rows", [((1, 1), 1), ((5, 300), 1), ((3, 7, 264), 1), ((1, 1), 128),
                                              ((2, 200, 264), 128), ((3, 2, 130, 77), 128), ((128, 128), 128)])
def test_quantize(dtype, shape, block_rows):
    x = (randn(*shape, seed=5) * torch.exp(randn(*shape[:-1], 1, seed=6))).to(dtype)
    x.view(-1, shape[-1])[0, : min(128, shape[-1])] = 0
    q = torch.empty(shape, dtype=F8, device="cuda")
    rows = shape[-2] if block_rows == 1 else R.nblk(shape[-2])
    s = torch.empty(*shape[:-2], rows, R.nblk(shape[-1]), device="cuda")
    moe.quantize_fp8(x, q, s, block_rows)
    v = x.double()
    _, want, half = R.quantize(v, block_rows)
    assert ((s.double() - want).abs() <= want * 2 * U32).all()
    err = (R.wide(q, s, block_rows) - v).abs()
    assert (err <= torch.maximum(half, v.abs() * 2.0 ** -4) * (1 + 1e-4) + v.abs() * 8 * U32).all()


# ------------------------------------------------------------------- select
def check_select(logits, K, norm, **o):
    T = logits.shape[0]
    sel = torch.full((T, K), -7, dtype=torch.int64, device="cuda")
    w = torch.full((T, K), NAN, device="cuda")
    moe.select_experts(logits, K, norm, sel, w, **o)
    want, ww = R.select(logits, K, norm, **o)
    assert torch.equal(sel, want)
    # scores: 20 steps (the exponent's rounding, 13 of the sum); the sum of the chosen: 8 more; 3 roundings
    assert ((w.double() - ww).abs() <= ww.abs() * 40 * U32 + 1e-37).all()


OPTS = [dict(), dict(score="sigmoid"), dict(groups=4, top_groups=2), dict(groups=2, top_groups=1, group_score="top2"),
        dict(score="sigmoid", groups=4, top_groups=3, group_score="top2", scale=2.5)]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("o", OPTS, ids=str)
@pytest.mark.parametrize("T,E", [(1, 4), (2, 8), (3, 12), (65, 20), (257, 32), (100, 64), (31, 100), (33, 128),
                                 (40, 160), (129, 252), (5000, 256)])
def test_select(T, E, o, bias):
    l = randn(T, E, seed=E, std=2.0)
    b = 0.1 * randn(E, seed=9) if bias else None
    most = E // o.get("groups", 1) * o.get("top_groups", 1)
    for K in {1, min(8, most), most if T < 100 else 1}:
        check_select(l, K, K % 2 == 0, selection_bias=b, **o)


@pytest.mark.parametrize("E,groups,top", [(6, 3, 2), (15, 5, 2), (252, 63, 10), (256, 256, 9), (256, 16, 3), (256, 32, 5),
                                          (96, 3, 1), (64, 64, 64)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_select_group_layouts(E, groups, top, score, group_score):
    o = dict(score=score, groups=groups, top_groups=top, group_score=group_score)
    l = randn(77, E, seed=E)
    check_select(l, min(6, top * (E // groups)), True, **o)
    check_select(l, min(6, top * (E // groups)), False, selection_bias=randn(E, seed=3), **o)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("o", OPTS, ids=str)
def test_select_near_and_equal_scores(o, bias):
    """Scores one rounding apart and exactly equal ones: the choice is that of 64 bits, ties to the lower index."""
    T, E = 600, 64
    l = randn(T, 1, seed=1) + torch.randint(-3, 4, (T, E), generator=gen(2), device="cuda") * 1e-7
    l[:200] = torch.randint(-2, 3, (200, E), generator=gen(3), device="cuda").float()
    l[200:250] = 0.0
    b = torch.randint(-2, 3, (E,), generator=gen(4), device="cuda") * 3e-8 if bias else None
    check_select(l, 4, True, selection_bias=b, **o)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("o", OPTS, ids=str)
def test_select_masked_and_not_finite(o, bias):
    T, E = 64, 32
    l = randn(T, E, seed=1)
    l[torch.rand(T, E, generator=gen(2), device="cuda") < 0.7] = -INF
    l[0] = -INF                                  # nothing left
    l[1] = torch.finfo(torch.float32).min
    l[2, :] = NAN
    l[3, 5], l[3, 9] = NAN, INF
    l[4, 31] = 3.0e38
    b = None
    if bias:
        b = 0.1 * randn(E, seed=3)
        b[::5] = -INF                            # experts switched off
    check_select(l, 6, True, selection_bias=b, **o)
    check_select(l, 6, False, selection_bias=b, **o)


@pytest.mark.parametrize("E,groups", [(256, 8), (64, 8), (250, 10)])       # groups as runs of lanes, and any size
@pytest.mark.parametrize("offset", [0.0, 100.0, 1000.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_group_candidates_few_ulps_apart(E, groups, offset, score):
    """The two best of a group among several that differ in their last bits, far from zero."""
    T, size = 400, E // groups
    ulp = 2.0 ** -14 if offset else 2.0 ** -23
    l = offset - 100.0 + torch.zeros(T, groups, size, device="cuda")
    n = min(size, 6)
    near = torch.randint(0, 16, (T, groups, n), generator=gen(1), device="cuda") * ulp
    l[:, :, :n] = offset + near.to(torch.float32)
    l[0] = offset - 100.0
    l[0, 0, :3] = torch.tensor([offset, offset, offset + 7 * ulp], device="cuda")
    l[0, 1, :2] = torch.tensor([offset + 0.01, offset - 0.0099], device="cuda")
    for top in (1, groups // 2):
        check_select(l.view(T, E), 2, False, score=score, groups=groups, top_groups=top, group_score="top2")


@pytest.mark.parametrize("E,groups", [(64, 32), (60, 30), (256, 8), (250, 10)])       # groups as runs of lanes, and any size
@pytest.mark.parametrize("size", [1.0, 10.0, 100.0, 1000.0, 1e38])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_group_sums_that_cancel(E, groups, size, score):
    """Biases of opposite signs whose sums lie near each other: a sum's error is that of its terms."""
    n = E // groups
    for seed in range(30):
        b = torch.full((groups, n), -4.0 * min(size, 5e37), device="cuda")
        b[:, 0] = size * (1 + 0.05 * torch.rand(groups, generator=gen(seed), device="cuda"))
        b[:, 1] = torch.randint(0, 8, (groups,), generator=gen(seed + 50), device="cuda") * 2e-7 * size - b[:, 0]
        l = randn(200, E, seed=seed, std=1e-6)
        check_select(l, 2, False, score=score, selection_bias=b.view(-1), groups=groups, top_groups=1 + seed % (groups - 1),
                     group_score="top2")


def test_select_group_sums_that_cancel_by_truncation():
    """All scores 1: 5 + 15 u - 5 is more than 5 + 21 u - 5 - 7 u, u = 2^-21."""
    u = 2.0 ** -21
    b = torch.full((64,), -20.0, device="cuda")
    b[:2] = torch.tensor([4 + 15 * u, -6.0])
    b[8:10] = torch.tensor([4 + 21 * u, -6.0 - 7 * u])
    l = torch.full((3, 64), 100.0, device="cuda")
    check_select(l, 2, False, score="sigmoid", selection_bias=b, groups=8, top_groups=1, group_score="top2")
    b2 = torch.zeros(4, device="cuda")
    b2[:] = torch.tensor([100.536850, -99.380936, 100.033401, -98.877495])
    b2 = torch.cat([b2, torch.full((60,), -300.0, device="cuda")])
    check_select(torch.zeros(3, 64, device="cuda"), 2, False, score="sigmoid", selection_bias=b2, groups=32, top_groups=1,
                 group_score="top2")


@pytest.mark.parametrize("E,groups", [(256, 8), (250, 10), (64, 32)])
@pytest.mark.parametrize("o", [dict(), dict(group_score="top2"), dict(score="sigmoid", group_score="top2")], ids=str)
@pytest.mark.parametrize("by_bias", [False, True])
def test_select_whole_groups_masked(E, groups, o, by_bias):
    """Groups of which nothing, one expert or two are left, kept and dropped; sums that pass fp32's range."""
    n = E // groups
    off = torch.zeros(groups, n, dtype=torch.bool, device="cuda")
    off[: groups // 2] = True
    off[0, 0] = off[1, : min(n, 2)] = False
    for extreme in (False, True):
        l, b = randn(90, E, seed=E), 0.1 * randn(E, seed=3)
        if by_bias:
            b[off.view(-1)] = -INF
            if extreme:
                b.view(groups, n)[1::3] = -3e38
                b.view(groups, n)[2::3] = 3e38
        else:
            l[:, off.view(-1)] = -INF
            b = None
        for top in (1, groups // 2, groups // 2 + 1, groups - 1):
            check_select(l, min(8, top * n), True, selection_bias=b, groups=groups, top_groups=top, **o)


def test_route_groups():
    """Both dtypes: the logits are the router's, the choice is that of select_experts on them."""
    for dtype, T, D, E in ((torch.bfloat16, 300, 264, 64), (torch.float32, 37, 33, 20)):
        x, r = randn(T, D, seed=1).to(dtype), randn(E, D, seed=2, std=0.1).to(dtype)
        rb = randn(E, seed=3)
        o = dict(score="sigmoid", selection_bias=randn(E, seed=4), groups=4, top_groups=2, group_score="top2")
        lg, lg2 = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
        sel, w = torch.empty(T, 5, dtype=torch.int64, device="cuda"), torch.empty(T, 5, device="cuda")
        moe.route_groups(x, r, 5, True, lg, sel, w, router_bias=rb, **o)
        s2, w2 = torch.empty_like(sel), torch.empty_like(w)
        moe.route(x, r, 5, True, s2, w2, router_bias=rb, router_logits=lg2)
        assert torch.equal(lg, lg2)
        want, _ = R.select(lg, 5, True, **o)
        assert torch.equal(sel, want)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("o", [dict(), dict(scale=2.5), dict(score="sigmoid"), dict(score="sigmoid", scale=0.5, groups=4,
                               top_groups=2, group_score="top2")], ids=str)
@pytest.mark.parametrize("dtype,T,D,E", [(torch.bfloat16, 300, 264, 64), (torch.float32, 37, 33, 20)], ids=str)
def test_route_groups_weights(dtype, T, D, E, o, norm):
    """What route_groups writes is what select_experts makes of its logits, and right against 64 bits."""
    x, r = randn(T, D, seed=1).to(dtype), randn(E, D, seed=2, std=0.1).to(dtype)
    for bias in (None, randn(E, seed=4)):
        lg = torch.empty(T, E, device="cuda")
        sel, w = torch.empty(T, 5, dtype=torch.int64, device="cuda"), torch.empty(T, 5, device="cuda")
        moe.route_groups(x, r, 5, norm, lg, sel, w, selection_bias=bias, **o)
        s2, w2 = torch.empty_like(sel), torch.empty_like(w)
        moe.select_experts(lg, 5, norm, s2, w2, selection_bias=bias, **o)
        assert torch.equal(sel, s2) and torch.equal(w, w2)
        check_select(lg, 5, norm, selection_bias=bias, **o)


# ------------------------------------------------------------------ product
def check_product(E, M, N, K, offsets, dtype=torch.bfloat16, seed=0):
    a, sa = rows8(M, K, seed)
    w, sw = weight8(E, N, K, seed + 10)
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    o = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    moe.gemm_fp8(a, sa, w, sw, out, offsets=o)
    C, S, live = R.product(a, sa, w, sw, offsets or [0, M])
    # 128 products a block (one step each if the tensor core truncates), a scaled sum per block, two scale products
    gamma = (128 + R.nblk(K) + 4) * 2 * U32
    err = (out.double() - C).abs()
    assert (err[live] <= (S * gamma + C.abs() * HALF[dtype] * 1.01)[live]).all()
    assert (out[~live] == 7.0).all()
    again = torch.full_like(out, 7.0)
    moe.gemm_fp8(a, sa, w, sw, again, offsets=o)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 256, 128), (7, 136, 144), (8, 264, 272), (9, 248, 4096),
                                   (33, 512, 1040), (100, 1000, 336), (128, 256, 512), (129, 392, 640),
                                   (300, 2056, 2064), (1000, 128, 128), (2, 4096, 7168)])
def test_product_dense(M, N, K, dtype):
    check_product(1, M, N, K, None, dtype)


@pytest.mark.parametrize("E,M,N,K,offsets", [
    (4, 300, 264, 272, [0, 0, 129, 129, 300]),           # empty experts first and in the middle
    (3, 50, 128, 128, [0, 0, 0, 0]),                     # no rows at all
    (3, 50, 136, 400, [5, 6, 30, 41]),                   # rows before the first and behind the last stay
    (2, 1, 40, 16, [0, 1, 1]),
    (5, 700, 520, 256, [0, 1, 9, 265, 640, 700]),
    (64, 640, 256, 512, list(range(0, 650, 10))),
    (256, 300, 72, 144, [min(300, 2 * i) for i in range(257)])])
def test_product_by_expert(E, M, N, K, offsets):
    check_product(E, M, N, K, offsets)
    check_product(E, M, N, K, offsets, torch.float32, seed=50)


def uneven(M, E, *rows):
    """Offsets of E experts over M rows: the given row counts first, the rest by turns."""
    o = [0]
    for r in rows:
        o.append(min(M, o[-1] + r))
    left = E - len(rows)
    return o + [o[-1] + (M - o[-1]) * (i + 1) // left for i in range(left)]


@pytest.mark.parametrize("E,M,N,K,offsets", [
    (1, 16, 24, 4096, None),                             # few tiles: the K blocks over a cluster
    (3, 70, 40, 2064, [0, 33, 33, 70]),
    (64, 1500, 264, 272, uneven(1500, 64, 3, 1400)),     # 32-row tiles, most of them one expert's
    (8, 800, 2056, 144, uneven(800, 8, 1, 0, 700)),
    (8, 5000, 304, 144, uneven(5000, 8, 0, 2500, 129)),  # 128-row tiles, more than 16 row blocks of an expert
    (2, 2000, 520, 400, [3, 903, 1990]),                 # pairs of CTAs with tails; rows around them stay
    (2, 1600, 264, 272, [0, 1, 1600]),
    (3, 2400, 128, 128, [0, 0, 2400, 2400]),
    (1, 4500, 600, 144, None)], ids=lambda v: "list" if isinstance(v, list) else str(v))
def test_product_row_forms(E, M, N, K, offsets):
    check_product(E, M, N, K, offsets, seed=3)
    check_product(E, M, N, K, offsets, torch.float32, seed=60)


def test_products_at_once():
    """Calls on two streams at the same time, each form with itself and with another."""
    args = []
    for i, (E, M, N, K) in enumerate([(1, 16, 256, 4096), (1, 16, 256, 4096), (4, 400, 512, 512), (2, 2000, 512, 512)]):
        a, sa = rows8(M, K, i)
        w, sw = weight8(E, N, K, i + 10)
        o = torch.tensor(uneven(M, E), dtype=torch.int32, device="cuda")
        args.append((a, sa, w, sw, o))
    outs = [torch.empty(x[0].shape[0], x[2].shape[1], device="cuda") for x in args]
    want = [torch.empty_like(o) for o in outs]
    for x, o in zip(args, want):
        moe.gemm_fp8(*x[:4], o, offsets=x[4])
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in args]
    for _ in range(20):
        for x, o, st in zip(args, outs, s):
            moe.gemm_fp8(*x[:4], o, offsets=x[4], stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_pair_products_back_to_back():
    """CTA pairs of one short tile, launched without a pause: each ends with nothing of its own still on the way."""
    a, sa = rows8(800, 16, 1)
    w, sw = weight8(1, 2048, 16, 2)
    want = torch.empty(800, 2048, device="cuda")
    moe.gemm_fp8(a, sa, w, sw, want)
    C, S, _ = R.product(a, sa, w, sw, [0, 800])
    assert ((want.double() - C).abs() <= S * 133 * 2 * U32 + C.abs() * U32 * 1.01).all()       # as in check_product
    outs = [torch.empty_like(want) for _ in range(4)]
    for i in range(400):
        moe.gemm_fp8(a, sa, w, sw, outs[i % 4])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_product_offsets_out_of_order_are_clamped():
    """Offsets beyond M count as M, descending ones as the one before."""
    a, sa = rows8(40, 128, 1)
    w, sw = weight8(3, 64, 128, 2)
    out = torch.zeros(40, 64, dtype=torch.float32, device="cuda")
    moe.gemm_fp8(a, sa, w, sw, out, offsets=torch.tensor([-5, 20, 10, 900], dtype=torch.int32, device="cuda"))
    want = torch.zeros_like(out)
    moe.gemm_fp8(a, sa, w, sw, want, offsets=torch.tensor([0, 20, 20, 40], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, want) and bool(out.abs().sum() > 0)


def test_product_zero_scales_and_nan_rows():
    """A NaN stays in its row; blocks of scale zero add nothing."""
    a, sa = rows8(70, 384, 1)
    w, sw = weight8(1, 136, 384, 2)
    a[9, 200] = NAN
    sa[:, 1] = 0.0
    sa[9, 1] = 1.0
    out = torch.empty(70, 136, device="cuda")
    moe.gemm_fp8(a, sa, w, sw, out)
    assert out[9].isnan().all() and not out[torch.arange(70, device="cuda") != 9].isnan().any()


# ------------------------------------------------------------------ experts
def make_experts(T, D, F, E, K, seed=0):
    x, xs = rows8(T, D, seed)
    gu = (randn(E, 2 * F, D, seed=seed + 2) * 100).clamp(-448, 448).to(F8)
    gus = (torch.rand(E, 2, R.nblk(F), R.nblk(D), generator=gen(seed + 3), device="cuda") + 0.5) / 100 / D ** 0.5
    dn, dns = weight8(E, D, F, seed + 4, std=F ** -0.5)
    sel = torch.rand(T, E, generator=gen(seed + 5), device="cuda").topk(K, 1).indices
    w = torch.rand(T, K, generator=gen(seed + 6), device="cuda")
    return [x, xs, sel, w, gu, gus, dn, dns]


def run_experts(args, stream=None):
    x, sel, dn = args[0], args[2], args[6]
    T, D = x.shape
    E, _, F = dn.shape
    ws = torch.full((moe.experts_workspace_size_fp8(T, D, F, E, sel.shape[1]),), 255, dtype=torch.uint8,
                    device="cuda")             # garbage: nothing of it may be relied on
    out = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    moe.experts_forward_fp8(*args, out, workspace=ws, stream=stream)
    return out


def check_experts(args, out):
    want, raw, bound = R.experts(*args)
    K = args[2].shape[1]
    # half a step of the intermediate's e4m3, each expert's rounding (to fp16 with a scale for 64 columns: 2^-11 of
    # the largest at most) and the sum's to bf16
    mag = want.abs() + bound
    each = sum((args[3][:, k:k + 1].double().abs() for k in range(K)))
    cap = raw.abs().amax(1, keepdim=True) + bound.amax(1, keepdim=True)
    tol = bound * 1.01 + mag * 2.0 ** -8 * 1.01 + each.clamp_min(1) * cap * 2.0 ** -7 + 1e-6
    assert ((out.double() - raw).abs() <= tol).all()
    # against the rounded intermediate: what is left are the two roundings (2^-8 each at most) and the few
    # values that fall on the other side of a border (a share of 1e-4, each 2^-4 off: 6e-4 in the norm)
    d = (out.double() - want).norm() / want.norm().clamp_min(1e-30)
    assert d <= 2.0 ** -8 + 2.0 ** -8 + 1e-3, float(d)


@pytest.mark.parametrize("T,D,F,E,K", [(1, 16, 16, 1, 1), (1, 256, 384, 8, 2), (3, 144, 272, 4, 4), (32, 512, 1408, 64, 6),
                                       (5, 128, 128, 256, 8), (200, 272, 400, 8, 2), (700, 256, 128, 4, 3),
                                       (2100, 128, 144, 64, 2), (129, 1024, 256, 1, 1)])
def test_experts(T, D, F, E, K):
    args = make_experts(T, D, F, E, K)
    out = run_experts(args)
    check_experts(args, out)
    assert torch.equal(out, run_experts(args))


@pytest.mark.parametrize("T,D,F,E,K", [(1, 2048, 1152, 2, 1), (3, 2064, 1040, 4, 2),     # K blocks over a cluster
                                       (600, 256, 400, 8, 2), (2100, 128, 144, 8, 2),      # 128-row tiles
                                       (2, 128, 144, 256, 192), (600, 128, 144, 64, 6), (512, 128, 144, 256, 8), (64, 144, 144, 64, 6), (77, 128, 144, 64, 5), (48, 128, 128, 256, 8),   # 384, 385 slots
                                       (1700, 256, 272, 4, 2), (4700, 144, 144, 2, 1)])    # pairs of CTAs
def test_experts_row_forms(T, D, F, E, K):
    args = make_experts(T, D, F, E, K, seed=40)
    out = run_experts(args)
    check_experts(args, out)
    args[2][:, 0] = E - 1                        # nearly all to one expert, some slots twice
    args[2][::7] = -1
    check_experts(args, run_experts(args))
    assert (run_experts(args)[::7] == 0).all()


@pytest.mark.parametrize("slots", [0, 2])           # the last sorted by one CTA, and the first that is not
@pytest.mark.parametrize("E", [4, 8, 64, 128, 256])
def test_experts_permutations(E, slots):
    """1800 + 20 E slots, 4096 at most; unevenly filled, some unused."""
    T = (min(1800 + 20 * E, 4096) + slots) // 2
    args = make_experts(T, 128, 128, E, 2, seed=30)
    args[2][: T // 2, 0] = 1
    args[2][::5, 1] = -1
    check_experts(args, run_experts(args))


def test_experts_at_once():
    """Two calls on two streams at the same time, a workspace each."""
    args = [make_experts(24, 512, 384, 8, 2, seed=1), make_experts(300, 256, 384, 8, 2, seed=2)]
    want = [run_experts(a) for a in args]
    ws = [torch.empty(moe.experts_workspace_size_fp8(*a[0].shape, 384, 8, 2), dtype=torch.uint8, device="cuda") for a in args]
    out = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in args]
    for _ in range(20):
        for a, o, w, st in zip(args, out, ws, s):
            moe.experts_forward_fp8(*a, o, workspace=w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(out, want))


@pytest.mark.parametrize("T", [7, 400])
def test_experts_unused_slots_and_repeats(T):
    """Slots outside [0, E) add nothing whatever their weight; a repeated expert counts twice; all to one expert."""
    args = make_experts(T, 256, 272, 8, 3, seed=20)
    sel, w = args[2], args[3]
    sel[0] = -1                                  # a padded token
    w[0] = NAN
    sel[1, 1], w[1, 1] = 8, INF
    sel[2] = sel[2, 0]
    sel[3, 2] = 2 ** 40
    out = run_experts(args)
    assert (out[0] == 0).all()
    args[3] = torch.where((sel < 0) | (sel >= 8), torch.zeros_like(w), w)
    check_experts(args, out)
    sel[:] = 5
    check_experts(args, run_experts(args))
    sel[:] = -1
    assert (run_experts(args) == 0).all()


@pytest.mark.parametrize("T", [2, 300, 1600])
def test_experts_infinite_column(T):
    """A column whose sum passes fp32's range is infinite; its neighbours keep their large finite values."""
    D, F = 256, 128
    x, xs, sel, w, gu, gus, dn, dns = make_experts(T, D, F, 2, 1, seed=5)
    x.copy_(torch.ones_like(x, dtype=torch.float32).to(F8))
    xs.fill_(1.0)
    gu.copy_(torch.ones_like(gu, dtype=torch.float32).to(F8))
    gus.fill_(1.0 / 32)                          # gate = up = 8: h about 64 in every column
    dn.copy_(torch.full_like(dn, 2.0 ** -6, dtype=torch.float32).to(F8))
    dn[:, 17] = 448.0
    dns.fill_(2.0 ** 110)
    w.fill_(1.0)
    out = run_experts([x, xs, sel, w, gu, gus, dn, dns])
    h = 8 / (1 + torch.exp(torch.tensor(-8.0, dtype=torch.float64))) * 8
    assert (out[:, 17] == INF).all()             # 128 * 64 * 448 * 2^110 > 2^128
    rest = out[:, torch.arange(D, device="cuda") != 17].double()
    want = float(h) * 128 * 2.0 ** 104
    # the intermediate's e4m3 (2^-4), fp16 and bf16
    assert ((rest / want - 1).abs() <= 2.0 ** -4 + 2.0 ** -7).all()


@pytest.mark.parametrize("T", [3, 300, 1000])       # 32-row tiles, 128-row tiles, pairs of CTAs
def test_experts_round_ties_of_the_intermediate_to_even(T):
    """h / scale halfway between two e4m3 values, in blocks whose scale's rounded reciprocal would end above the tie."""
    r = torch.arange(1, 4096, 2, dtype=torch.float32)
    above = (48 * r) * (1 / ((64 * r) / 448)) > 336             # 336 of 448 lies halfway between 320 and 352
    r = r[above][:40]
    D, F, n = 128, 40 * 128, len(r)
    assert n == 40
    x = torch.zeros(T, D, device="cuda")
    x[:, 0] = 1.0
    gu = torch.zeros(1, 2, F, D, device="cuda")
    gu[0, 0, :, 0] = 64.0                                       # silu(64) = 64 in fp32
    gu[0, 1, :, 0] = 0.75                                       # h = 48 r,
    gu[0, 1, ::128, 0] = 1.0                                    # and once in each block 64 r, the largest
    gus = torch.ones(1, 2, n, 1, device="cuda")
    gus[0, 1, :, 0] = r.cuda()
    dn = torch.zeros(1, D, F, device="cuda")
    d = torch.arange(D, device="cuda")
    dn[0, d, 128 * (d % n) + 1 + d // n] = 1.0
    out = run_experts([x.to(F8), torch.ones(T, 1, device="cuda"), torch.zeros(T, 1, dtype=torch.int64, device="cuda"),
                       torch.ones(T, 1, device="cuda"), gu.view(1, 2 * F, D).to(F8), gus, dn.to(F8),
                       torch.ones(1, 1, n, device="cuda")])
    want = 320 / 448 * 64 * r.cuda().double()[d % n]            # to even
    assert ((out.double() / want - 1).abs() <= 2.0 ** -8 + 2.0 ** -11 + 4 * U32).all()     # bf16, fp16, the scale


@pytest.mark.parametrize("cancel", [False, True])
@pytest.mark.parametrize("T,D,F,E", [(3, 512, 256, 2), (40, 1024, 1152, 8),            # 32-row tiles, K blocks over a cluster or not
                                     (700, 1088, 384, 4), (2000, 512, 256, 2)])        # 128-row tiles, pairs of CTAs
def test_experts_outputs_are_kept_to_fp16(T, D, F, E, cancel):
    """An intermediate that 8 bits hold exactly, so that only each expert's fp16 and the sum's bf16 are left: column
    blocks far apart in size, and experts that cancel, where bf16 for each expert's output would be 8 times as far off."""
    K = 2
    up = (randn(E, F, D, seed=1) * 100).clamp(-448, 448).to(F8)
    up.view(torch.uint8)[:, ::128] = 0x7E        # 448 in every block: the scale is a power of two
    gu = torch.stack([torch.full_like(up, 64.0, dtype=torch.float32).to(F8), up], 1).view(E, 2 * F, D)     # silu(64) = 64
    gus = torch.ones(E, 2, R.nblk(F), R.nblk(D), device="cuda")
    size = torch.where(torch.arange(D, device="cuda") // 64 % 2 == 0, 2.0 ** 6, 2.0 ** -5)     # 2^11 apart
    dn = (randn(E, D, F, seed=2) * size[:, None]).clamp(-448, 448).to(F8)
    dns = torch.exp2(torch.randint(-12, 12, (E, R.nblk(D), R.nblk(F)), generator=gen(3), device="cuda").float())
    sel = torch.rand(T, E, generator=gen(4), device="cuda").topk(K, 1).indices
    w = torch.rand(T, K, generator=gen(5), device="cuda") + 0.1
    if cancel:
        less = randn(E // 2, D, F, seed=6) > 2
        dn[1::2] = torch.where(less, torch.zeros((), device="cuda"), -dn[::2].float()).to(F8)
        dns[1::2] = dns[::2]
        sel = sel[:, :1] // 2 * 2 + torch.tensor([0, 1], device="cuda")
        w = w[:, :1].expand(T, K).contiguous()
    at = torch.arange(T, device="cuda") % D
    x = torch.zeros(T, D, device="cuda")
    x[torch.arange(T, device="cuda"), at] = 1.0
    out = run_experts([x.to(F8), torch.ones(T, R.nblk(D), device="cuda"), sel, w, gu, gus, dn, dns]).double()
    W = R.wide(dn, dns, R.BLOCK)
    want, tol, coarse = (torch.zeros(T, D, dtype=torch.float64, device="cuda") for _ in range(3))
    for e in range(E):
        t, k = (sel == e).nonzero(as_tuple=True)
        h = 64 * up[e].double()[:, at[t]].T
        y, S, we = h @ W[e].T, h.abs() @ W[e].abs().T, w[t, k].double()[:, None]
        cap = torch.nn.functional.pad(y.abs(), (0, -D % 64)).unflatten(1, (-1, 64)).amax(-1).repeat_interleave(64, 1)[:, :D]
        want.index_add_(0, t, we * y)
        coarse.index_add_(0, t, we * y.bfloat16().double())
        # fp16: half a step of 2^-10 (of 2^-24 below 2^-14, with the block's largest at 2^14); the products' sums
        # as in check_product; the weighted sum's K products and additions
        tol.index_add_(0, t, we * (y.abs() * (2.0 ** -11 + 4 * U32) + cap * 2.0 ** -39 + S * (128 + R.nblk(F) + 4) * 2 * U32))
    tol += (want.abs() + tol) * 2.0 ** -8
    assert ((out - want).abs() <= tol).all()
    if cancel:                                   # bf16 outputs would be seen
        assert ((coarse - want).abs() > tol).double().mean() > 0.02


def test_experts_streams_graph_and_shared_workspace():
    """Another stream; two captured calls that share a workspace, replayed with new inputs."""
    args, other = make_experts(24, 256, 384, 8, 2, seed=1), make_experts(300, 256, 384, 8, 2, seed=2)
    want, want2 = run_experts(args), run_experts(other)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert torch.equal(run_experts(args), want)
    s.synchronize()
    ws = torch.empty(max(moe.experts_workspace_size_fp8(T, 256, 384, 8, 2) for T in (24, 300)), dtype=torch.uint8,
                     device="cuda")
    out, out2 = torch.empty_like(want), torch.empty_like(want2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.experts_forward_fp8(*args, out, workspace=ws)
        moe.experts_forward_fp8(*other, out2, workspace=ws)
    for _ in range(2):
        out.zero_(), out2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, want2)
    fresh = make_experts(24, 256, 384, 8, 2, seed=7)
    for a, b in zip(args, fresh):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, run_experts(fresh))


def test_small_calls_capture():
    """The norm, the choice and the product in one graph."""
    x, r, w = randn(9, 256, seed=1).bfloat16(), randn(9, 256, seed=2).bfloat16(), randn(256, seed=3).bfloat16()
    want = run_norm(x, r, w, 1e-6)
    wt, sw = weight8(1, 64, 256, 4)
    lg = randn(9, 64, seed=5)
    o = run_norm(x, r, w, 1e-6)
    out, ref = torch.empty(9, 64, device="cuda"), torch.empty(9, 64, device="cuda")
    sel, ww = torch.empty(9, 4, dtype=torch.int64, device="cuda"), torch.empty(9, 4, device="cuda")

    def step(dst):
        moe.add_rmsnorm(x, w, 1e-6, residual=r, **o)
        moe.gemm_fp8(o["out8"], o["scales"], wt, sw, dst)
        moe.select_experts(lg, 4, True, sel, ww)

    step(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out)
    for v in o.values():
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k].view(torch.uint8), want[k].view(torch.uint8)) for k in o)
    assert torch.equal(out, ref) and torch.equal(sel, R.select(lg, 4, True)[0])


def test_profiler_counts_the_call():
    args = make_experts(16, 256, 256, 4, 2)
    run_experts(args)
    moe.profile_enable(True)
    run_experts(args)
    run_experts(args)
    ms, calls = moe.profile_read()
    moe.profile_enable(False)
    assert calls == 2
    assert all(ms[k] > 0 for k in ("permute", "gate_up", "down", "combine")) and ms["router"] == 0


# -------------------------------------------------------------------- block
@pytest.mark.parametrize("T,D,F,E,K,residual", [(1, 256, 384, 16, 4, True), (77, 272, 400, 16, 4, True),
                                                (600, 256, 256, 8, 2, False)])
def test_block(T, D, F, E, K, residual):
    """Norm, routing with groups and experts together, each step against float64 on what the step before gave."""
    bf = torch.bfloat16
    router, gu = randn(E, D, seed=1, std=0.1).to(bf), randn(E, 2 * F, D, seed=2, std=D ** -0.5).to(bf)
    dn = randn(E, D, F, seed=3, std=F ** -0.5).to(bf)
    nw = (1 + 0.1 * randn(D, seed=4)).to(bf) if residual else None
    o = dict(score="sigmoid", selection_bias=0.1 * randn(E, seed=5), groups=4, top_groups=2, group_score="top2", scale=2.5)
    blk = moe.MoEBlockFP8(router, gu, dn, top_k=K, norm_weight=nw, **o)
    x, r = randn(T, D, seed=6).to(bf), randn(T, D, seed=7).to(bf)
    out = blk(x, r) if residual else blk(x)
    y, y64 = x, x.double()
    if residual:
        h, y64 = R.add_rmsnorm(x, r, nw, 1e-6)
        assert torch.equal(blk.residual_, h)
        y = y64.to(bf)
    lg = y.double() @ router.double().T
    assert ((blk.router_logits_.double() - lg).abs() <= (y.double().abs() @ router.double().abs().T) * 2.0 ** -7).all()
    sel, w = R.select(blk.router_logits_, K, True, **o)
    assert torch.equal(sel, blk.selected_experts_)
    # the layer in 64 bits on unrounded weights: 8-bit values are off by 2^-4 at most each (2^-5 to 2^-6 on average,
    # independent); of x, gate, up, h and down together under 2^-3 in the norm
    X = y64
    want = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for k in range(K):
        g, u = (torch.einsum("td,tfd->tf", X, gu.view(E, 2, F, D)[sel[:, k], i].double()) for i in (0, 1))
        want += w[:, k:k + 1] * torch.einsum("tf,tdf->td", g * torch.sigmoid(g) * u, dn[sel[:, k]].double())
    assert (out.double() - want).norm() <= 2.0 ** -3 * want.norm()
    again = blk(x, r) if residual else blk(x)
    assert torch.equal(out, again)


def make_block(E=16, D=256, F=384):
    bf = torch.bfloat16
    return moe.MoEBlockFP8(randn(E, D, seed=1, std=0.1).to(bf), randn(E, 2 * F, D, seed=2, std=D ** -0.5).to(bf),
                           randn(E, D, F, seed=3, std=F ** -0.5).to(bf), top_k=4, norm_weight=(1 + 0.1 * randn(D, seed=4)).to(bf),
                           score="sigmoid", groups=4, top_groups=2)


def test_block_on_streams_at_once():
    """One block on two streams (an object and a raw handle) at the same time."""
    blk = make_block()
    xs = [randn(T, 256, seed=T).bfloat16() for T in (40, 700)]
    want = [blk(x, x) for x in xs]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        got = [blk(x, x, stream=st if i else st.cuda_stream) for i, (x, st) in enumerate(zip(xs, s))]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_block_is_ready_when_made():
    """Its weights are in place on return, so that a first call on another stream needs no wait."""
    make_block()                                 # kernels are loaded by their first launch, which waits for the device
    a = randn(8192, 8192, seed=1)
    for _ in range(30):
        a @ a                                    # some 500 ms for the quantiser to queue behind
    blk = make_block()
    assert torch.cuda.current_stream().query()
    x = randn(40, 256, seed=2).bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(blk(x, x, stream=s), blk(x, x))


def test_block_in_two_threads():
    """One block, two threads with a stream and tokens of their own, as many of them in each."""
    blk = make_block()
    xs = [randn(60, 256, seed=s).bfloat16() for s in (1, 2)]
    want = [blk(x, x) for x in xs]
    torch.cuda.synchronize()
    bad = [None, None]

    def calls(i):
        st = torch.cuda.Stream()
        wrong = 0
        for _ in range(100):
            got = blk(xs[i], xs[i], stream=st)
            st.synchronize()                     # the comparison runs on the default stream
            wrong += not torch.equal(got, want[i])
        bad[i] = wrong

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == [0, 0]


def test_block_captured_twice():
    """Two graphs of one block, replayed at the same time with an eager call, and again with other inputs."""
    blk = make_block()
    xs = [randn(T, 256, seed=T).bfloat16() for T in (40, 700, 300)]
    want = [blk(x, x) for x in xs]
    graphs, outs = [], []
    for x in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(blk(x, x))
        graphs.append(g)
    s = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, s):
            with torch.cuda.stream(st):
                g.replay()
        eager = blk(xs[2], xs[2])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([*outs, eager], want))
    xs[0].copy_(randn(40, 256, seed=99))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], blk(xs[0], xs[0]))


# ----------------------------------------------------- beyond the small cases
def test_product_offsets_at_four_bytes():
    a, sa = rows8(90, 272, 1)
    w, sw = weight8(3, 72, 272, 2)
    out, want = torch.zeros(90, 72, device="cuda"), torch.zeros(90, 72, device="cuda")
    o = torch.tensor([7, 0, 30, 41, 90], dtype=torch.int32, device="cuda")
    moe.gemm_fp8(a, sa, w, sw, out, offsets=o[1:])
    moe.gemm_fp8(a, sa, w, sw, want, offsets=o[1:].clone())
    assert torch.equal(out, want) and bool(out.abs().sum() > 0)


@pytest.mark.parametrize("T", [40, 900, 30000])        # slots sorted by gate_up, by one CTA, and over many
def test_dependent_launch_setting_changes_nothing(T):
    args = make_experts(T, 128, 144, 8, 2, seed=3)
    want = run_experts(args)
    before = moe.set_pdl(True)
    try:
        for _ in range(3):
            assert torch.equal(run_experts(args), want)
    finally:
        moe.set_pdl(before)


def test_debug_sync_gives_the_same():
    args = make_experts(40, 256, 384, 8, 2, seed=3)
    want = run_experts(args)
    before = moe.set_debug_sync(5000)
    try:
        assert torch.equal(run_experts(args), want)
    finally:
        moe.set_debug_sync(before)


def test_norm_past_32_bits():
    T, D = 270_000, 8192                          # 2.2e9 elements
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(1))
    w = (1 + 0.3 * randn(D, seed=3)).bfloat16()
    o = run_norm(x, None, w, 1e-6, sum_out=False)
    check_norm(x[-3:], None, w, 1e-6, {k: v if v is None else v[-3:] for k, v in o.items()})


def test_select_past_32_bits():
    T, E = 8_400_000, 256                         # 2.15e9 logits
    lg = torch.empty(T, E, device="cuda").normal_(generator=gen(1))
    sel, w = torch.empty(T, 8, dtype=torch.int64, device="cuda"), torch.empty(T, 8, device="cuda")
    moe.select_experts(lg, 8, True, sel, w, score="sigmoid", groups=8, top_groups=4, group_score="top2")
    for part in (slice(0, 2000), slice(T - 2000, T)):
        want, w64 = R.select(lg[part], 8, True, score="sigmoid", groups=8, top_groups=4, group_score="top2")
        assert torch.equal(sel[part], want)
        assert ((w[part].double() - w64).abs() <= 1e-6).all()


@pytest.mark.parametrize("M,N,K", [(70_000, 32_768, 128), (280_000, 64, 8192)])      # out, or a, passes 2^31 bytes
def test_product_past_32_bits(M, N, K):
    a = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(std=150, generator=gen(1)).clamp_(-448, 448).to(F8)
    sa = torch.rand(M, R.nblk(K), generator=gen(2), device="cuda") / 150
    w, sw = weight8(1, N, K, 3)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    moe.gemm_fp8(a, sa, w, sw, out)
    for part in (slice(0, 40), slice(M - 40, M)):
        C, S, _ = R.product(a[part], sa[part], w, sw, [0, 40])
        gamma = (128 + R.nblk(K) + 4) * 2 * U32       # as in check_product
        assert ((out[part].double() - C).abs() <= S * gamma + C.abs() * HALF[torch.bfloat16] * 1.01).all()


def test_experts_past_32_bits():
    """The intermediate and the experts' outputs pass 2^31 elements; first and last tokens against a call of their own."""
    T, D, F, E, K = 34_000, 8192, 8192, 8, 8
    args = make_experts(64, D, F, E, K, seed=9)
    big = [v.repeat((T // 64 + 1,) + (1,) * (v.dim() - 1))[:T].contiguous() if i < 4 else v for i, v in enumerate(
        [args[0].view(torch.uint8), *args[1:]])]
    big[0] = big[0].view(F8)
    out, few = run_experts(big), run_experts(args)
    for t in range(0, T, 64):
        n = min(64, T - t)
        if t and t + 128 < T:
            continue
        # the same values, added in another order and rounded to fp16 blocks and bf16
        d = (out[t:t + n].double() - few[:n].double()).abs()
        assert (d <= few[:n].double().abs() * 2.0 ** -7 + few[:n].double().abs().amax(1, keepdim=True) * 2.0 ** -9).all()
