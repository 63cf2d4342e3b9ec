"""MoEBlockFP8's host side, on the CPU: the calls it makes are replaced by ones
that record and hold up what they are given."""
import threading

import pytest

torch = pytest.importorskip("torch")

from mixture_experts_ffn_09_b200 import moe  # noqa: E402


def test_two_threads_keep_to_their_own_buffers(monkeypatch):
    """Both calls are inside each step at the same time, and each goes on with what its own steps wrote."""
    meet = threading.Barrier(2, timeout=30)

    def norm(x, w, eps, residual, sum_out, out, x8, xs):
        meet.wait()
        sum_out.copy_(x + residual)
        out.copy_(x)
        meet.wait()

    def route(x, router, K, norm_topk, logits, selected, weights, router_bias, **o):
        meet.wait()
        logits.fill_(float(x[0, 0]))
        selected.fill_(int(x[0, 0]))
        weights.fill_(float(x[0, 0]))
        meet.wait()

    def experts(x8, xs, selected, weights, *rest):
        meet.wait()
        rest[4].fill_(float(selected[0, 0]) + 100 * float(weights[0, 0]))
        meet.wait()

    monkeypatch.setattr(moe, "quantize_fp8", lambda *a: None)
    monkeypatch.setattr(moe, "add_rmsnorm", norm)
    monkeypatch.setattr(moe, "route_groups", route)
    monkeypatch.setattr(moe, "experts_forward_fp8", experts)
    monkeypatch.setattr(moe, "experts_workspace_size_fp8", lambda *a: 16)
    blk = moe.MoEBlockFP8(torch.zeros(4, 16), torch.zeros(4, 32, 16), torch.zeros(4, 16, 16), norm_weight=torch.ones(16))
    out = {}

    def call(i):
        out[i] = blk(torch.full((3, 16), float(i)), torch.full((3, 16), 0.5))

    threads = [threading.Thread(target=call, args=(i,)) for i in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in (1, 2):
        assert (out[i] == 101 * i).all()
    last = int(blk.selected_experts_[0, 0])
    assert last in (1, 2) and blk.residual_ is not None and blk.router_logits_.shape == (3, 4)
