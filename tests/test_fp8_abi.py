"""The 8-bit path's refusals, on the CPU: every call here fails host
validation, before anything is launched."""
import ctypes

import pytest

from mixture_experts_ffn_09_b200 import moe

P, MIS = 0x10000, 0x10008          # stand-ins for device pointers, never dereferenced


@pytest.fixture(scope="module")
def L():
    from mixture_experts_ffn_09_b200 import build
    build.build()
    return moe.lib()


def call(fn, kw, **change):
    kw = dict(kw, **change)
    return fn(*kw.values())


def opts(**kw):
    o = moe.GroupOpts(0, None, 0, 0, 0, 1.0)
    for k, v in kw.items():
        setattr(o, k, v)
    return ctypes.byref(o)


NORM = dict(x=P, residual=P, weight=P, eps=1e-6, T=4, D=64, dt=moe.BF16, sum_out=P, out=2 * P, q=P, scales=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(dt=moe.F64), moe.MOE_ERR_DTYPE), (dict(dt=17), moe.MOE_ERR_DTYPE),
    (dict(T=0), moe.MOE_ERR_INVALID_ARG), (dict(D=0), moe.MOE_ERR_INVALID_ARG), (dict(T=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(x=None), moe.MOE_ERR_INVALID_ARG), (dict(weight=None), moe.MOE_ERR_INVALID_ARG),
    (dict(out=None, q=None, scales=None), moe.MOE_ERR_INVALID_ARG), (dict(scales=None), moe.MOE_ERR_INVALID_ARG),
    (dict(q=None), moe.MOE_ERR_INVALID_ARG), (dict(out=P), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=-1.0), moe.MOE_ERR_INVALID_ARG), (dict(eps=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=float("inf")), moe.MOE_ERR_INVALID_ARG), (dict(D=32769), moe.MOE_ERR_SHAPE), (dict(T=2 ** 31), moe.MOE_ERR_SHAPE),
    (dict(x=MIS), moe.MOE_ERR_ALIGNMENT), (dict(residual=MIS), moe.MOE_ERR_ALIGNMENT), (dict(scales=MIS), moe.MOE_ERR_ALIGNMENT)])
def test_norm_refusals(L, change, want):
    assert call(L.moe_add_rmsnorm, NORM, **change) == want and moe.last_error()


QUANT = dict(x=P, dt=moe.F32, mats=1, rows=4, cols=4, block=1, q=P, scales=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(dt=moe.F64), moe.MOE_ERR_DTYPE), (dict(mats=0), moe.MOE_ERR_INVALID_ARG), (dict(rows=0), moe.MOE_ERR_INVALID_ARG),
    (dict(cols=-3), moe.MOE_ERR_INVALID_ARG), (dict(block=64), moe.MOE_ERR_INVALID_ARG), (dict(x=None), moe.MOE_ERR_INVALID_ARG),
    (dict(scales=None), moe.MOE_ERR_INVALID_ARG), (dict(rows=2 ** 31), moe.MOE_ERR_SHAPE),
    (dict(rows=2 ** 16, mats=2 ** 16), moe.MOE_ERR_SHAPE), (dict(cols=2 ** 31), moe.MOE_ERR_SHAPE),
    (dict(mats=2 ** 62, rows=4), moe.MOE_ERR_SHAPE), (dict(q=MIS), moe.MOE_ERR_ALIGNMENT)])
def test_quantize_refusals(L, change, want):
    assert call(L.moe_quantize_fp8, QUANT, **change) == want and moe.last_error()


SELECT = dict(logits=P, T=4, E=64, K=8, norm=1, opts=None, sel=P, w=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=0), moe.MOE_ERR_INVALID_ARG), (dict(E=0), moe.MOE_ERR_INVALID_ARG), (dict(K=0), moe.MOE_ERR_INVALID_ARG),
    (dict(K=65), moe.MOE_ERR_INVALID_ARG), (dict(E=257), moe.MOE_ERR_SHAPE), (dict(T=2 ** 31), moe.MOE_ERR_SHAPE),
    (dict(logits=None), moe.MOE_ERR_INVALID_ARG), (dict(sel=None), moe.MOE_ERR_INVALID_ARG), (dict(w=None), moe.MOE_ERR_INVALID_ARG),
    (dict(logits=MIS), moe.MOE_ERR_ALIGNMENT),
    (dict(opts=opts(score=2)), moe.MOE_ERR_INVALID_ARG), (dict(opts=opts(group_score=2)), moe.MOE_ERR_INVALID_ARG),
    (dict(opts=opts(groups=7)), moe.MOE_ERR_INVALID_ARG), (dict(opts=opts(groups=-1)), moe.MOE_ERR_INVALID_ARG),
    (dict(opts=opts(groups=4, top_groups=5)), moe.MOE_ERR_INVALID_ARG), (dict(opts=opts(top_groups=-1)), moe.MOE_ERR_INVALID_ARG),
    (dict(opts=opts(groups=16, top_groups=1)), moe.MOE_ERR_INVALID_ARG),       # K = 8 of 4 experts
    (dict(opts=opts(scale=float("nan"))), moe.MOE_ERR_INVALID_ARG), (dict(opts=opts(scale=float("inf"))), moe.MOE_ERR_INVALID_ARG),
    (dict(opts=opts(selection_bias=MIS)), moe.MOE_ERR_ALIGNMENT)])
def test_select_refusals(L, change, want):
    assert call(L.moe_select_experts, SELECT, **change) == want and moe.last_error()


ROUTE = dict(x=P, router=P, rb=None, T=4, D=64, E=64, K=8, norm=1, dt=moe.BF16, opts=None, logits=P, sel=P, w=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(dt=moe.F64), moe.MOE_ERR_DTYPE), (dict(D=0), moe.MOE_ERR_INVALID_ARG), (dict(D=2 ** 31), moe.MOE_ERR_SHAPE),
    (dict(D=60), moe.MOE_ERR_ALIGNMENT), (dict(x=None), moe.MOE_ERR_INVALID_ARG), (dict(logits=None), moe.MOE_ERR_INVALID_ARG),
    (dict(router=MIS), moe.MOE_ERR_ALIGNMENT), (dict(K=65), moe.MOE_ERR_INVALID_ARG), (dict(E=300), moe.MOE_ERR_SHAPE)])
def test_route_groups_refusals(L, change, want):
    assert call(L.moe_route_groups, ROUTE, **change) == want and moe.last_error()


GEMM = dict(a=P, sa=P, w=P, sw=P, offsets=P, E=4, M=32, N=64, K=64, out=P, dt=moe.BF16, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(dt=moe.F64), moe.MOE_ERR_DTYPE), (dict(E=0), moe.MOE_ERR_INVALID_ARG), (dict(M=0), moe.MOE_ERR_INVALID_ARG),
    (dict(N=0), moe.MOE_ERR_INVALID_ARG), (dict(K=0), moe.MOE_ERR_INVALID_ARG), (dict(a=None), moe.MOE_ERR_INVALID_ARG),
    (dict(sw=None), moe.MOE_ERR_INVALID_ARG), (dict(out=None), moe.MOE_ERR_INVALID_ARG), (dict(offsets=None), moe.MOE_ERR_INVALID_ARG),
    (dict(E=257), moe.MOE_ERR_SHAPE), (dict(M=2 ** 31), moe.MOE_ERR_SHAPE), (dict(N=2 ** 30), moe.MOE_ERR_SHAPE),
    (dict(K=2 ** 31), moe.MOE_ERR_SHAPE), (dict(E=1, M=2 ** 30, N=2 ** 30), moe.MOE_ERR_SHAPE),
    (dict(K=72), moe.MOE_ERR_ALIGNMENT), (dict(N=60), moe.MOE_ERR_ALIGNMENT), (dict(w=MIS), moe.MOE_ERR_ALIGNMENT),
    (dict(offsets=P + 2), moe.MOE_ERR_ALIGNMENT)])
def test_gemm_refusals(L, change, want):
    assert call(L.moe_gemm_fp8, GEMM, **change) == want and moe.last_error()


EXPERTS = dict(x=P, xs=P, sel=P, rw=P, gu=P, gus=P, dn=P, dns=P, out=P, T=4, D=64, F=64, E=8, K=2, ws=P, nb=1 << 40, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=0), moe.MOE_ERR_INVALID_ARG), (dict(F=0), moe.MOE_ERR_INVALID_ARG), (dict(K=9), moe.MOE_ERR_INVALID_ARG),
    (dict(K=0), moe.MOE_ERR_INVALID_ARG), (dict(E=300), moe.MOE_ERR_SHAPE), (dict(T=2 ** 30, K=2), moe.MOE_ERR_SHAPE),
    (dict(F=2 ** 28, E=8), moe.MOE_ERR_SHAPE), (dict(D=2 ** 26), moe.MOE_ERR_SHAPE), (dict(D=72), moe.MOE_ERR_ALIGNMENT), (dict(F=8), moe.MOE_ERR_ALIGNMENT),
    (dict(x=None), moe.MOE_ERR_INVALID_ARG), (dict(dns=None), moe.MOE_ERR_INVALID_ARG), (dict(out=MIS), moe.MOE_ERR_ALIGNMENT),
    (dict(ws=None), moe.MOE_ERR_WORKSPACE), (dict(nb=64), moe.MOE_ERR_WORKSPACE), (dict(ws=MIS), moe.MOE_ERR_ALIGNMENT)])
def test_experts_refusals(L, change, want):
    assert call(L.moe_experts_forward_fp8, EXPERTS, **change) == want and moe.last_error()


def test_experts_workspace_size(L):
    assert moe.experts_workspace_size_fp8(1, 64, 64, 8, 2) > 0
    for bad in ((0, 64, 64, 8, 2), (1, 65, 64, 8, 2), (1, 64, 64, 8, 9), (1, 64, 64, 300, 2)):
        assert moe.experts_workspace_size_fp8(*bad) == 0
    small, large = (moe.experts_workspace_size_fp8(T, 256, 512, 8, 2) for T in (16, 4096))
    assert small < large


def test_binding_refusals():
    """Shapes, types and devices are checked on the tensors before the call."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.add_rmsnorm(x, torch.zeros(64), 1e-6, out=torch.zeros(4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        moe.select_experts(x, 2, True, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))
    with pytest.raises(TypeError, match="dtype"):
        moe.select_experts(x.bfloat16(), 2, True, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))
    with pytest.raises(TypeError, match="dtype"):
        moe.gemm_fp8(x, x, x, x, x)
    with pytest.raises(ValueError, match="two dimensions"):
        moe.quantize_fp8(x[0], x[0], x[0])
    with pytest.raises(moe.MoEError) as e:
        moe.add_rmsnorm(x.double(), x[0].double(), 1e-6, out=x.double(), stream=0)
    assert e.value.status == moe.MOE_ERR_DTYPE
    with pytest.raises(ValueError, match="top_k"):
        moe.MoEBlockFP8(torch.zeros(4, 8), torch.zeros(4, 16, 8), torch.zeros(4, 8, 8), top_k=5)
