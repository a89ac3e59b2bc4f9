"""Buffers that a call on another stream makes.  They come from that stream's memory: a
block that the current stream has freed may still be in use there, and one that the call
drops must not go back to a stream that does not wait for it."""

import time

import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import api

pytestmark = pytest.mark.gpu

NEW, PRE, HQ, HKV, D = [40, 25], [30, 0], 4, 2, 64


def calls():
    """name -> call of the entry point with stream=..., all buffers left to it."""
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    N, KV = sum(NEW), sum(NEW) + sum(PRE)
    q, k, v = r(N, HQ, D), r(KV, HKV, D), r(KV, HKV, D)
    plan = cpa.make_plan(NEW, PRE, 2, "zigzag")
    segs = plan.segs[: plan.total_segs]
    segs_host = segs.cpu()
    o3 = torch.randn(3, N, HQ, D, generator=g, device="cuda")
    l3 = torch.randn(3, N, HQ, generator=g, device="cuda")
    shared = cpa.make_shared_plan([1] * N, [0] * N, KV, HQ, HKV)
    cache = cpa.alloc_kv_cache(KV, HKV, D, D)
    cpa.cp_kv_quantize(cache, k, v)
    return {
        "partial": lambda **kw: cpa.cp_attn_partial(segs, q, k, v, 0.1, **kw),
        "prefill": lambda **kw: cpa.cp_attn_prefill(segs, q, k, v, 0.1, **kw),
        "partial_restore": lambda **kw: cpa.cp_attn_partial_restore(segs, q, k, v, 0.1, plan.gather_idx, **kw),
        "merge": lambda **kw: cpa.cp_lse_merge(o3, l3, **kw),
        "restore": lambda **kw: (cpa.cp_restore(q, plan.restore_idx, **kw),),
        "partial_kv": lambda **kw: cpa.cp_attn_partial_kv(plan, q, k, v, 0.1, 32, **kw),
        "split_kv": lambda **kw: cpa.cp_attn_split_kv(segs, q, k, v, 0.1, 32, segs_host=segs_host, **kw),
        "pass_q": lambda **kw: cpa.cp_pass_q_attention(q, k, v, plan, 0.1, **kw),
        "prefill_attention": lambda **kw: cpa.cp_prefill_attention(q, k, v, plan, 0.1, **kw),
        "plan": lambda **kw: [getattr(cpa.make_plan(NEW, PRE, 2, "zigzag", **kw), n)
                              for n in ("segs", "tiles", "gather_idx", "positions", "restore_idx")],
        "shared": lambda **kw: cpa.cp_attn_shared(shared, q, k, v, 0.1, **kw),
        "kv_dequantize": lambda **kw: cpa.cp_kv_dequantize(cache, **kw),
    }


NAMES = ("partial", "prefill", "partial_restore", "merge", "restore", "partial_kv", "split_kv", "pass_q",
         "prefill_attention", "plan", "shared", "kv_dequantize")


@pytest.mark.parametrize("name", NAMES)
def test_buffers_belong_to_the_calls_stream(name, monkeypatch):
    call = calls()[name]
    want = [t.clone() for t in call() if t is not None]
    workspaces = [t.dtype == torch.uint8 for t in want]  # (hold what the call left there)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made, empty = [], torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        if t.is_cuda:
            made.append(torch.cuda.current_stream().cuda_stream)
        return t

    monkeypatch.setattr(api.torch, "empty", spy)
    got = [t for t in call(stream=side) if t is not None]
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert made and set(made) == {side.cuda_stream}
    for a, b, ws in zip(got, want, workspaces):
        assert ws or torch.equal(a, b)


def test_blocks_of_the_current_stream_are_not_taken():
    """The blocks that the current stream has just freed are not those that the shared-key
    attention and the cache's read-back get on another stream."""
    call = calls()
    run = lambda **kw: [*call["shared"](**kw), *call["kv_dequantize"](**kw)]  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    here = [torch.empty_like(t) for t in want for _ in range(3)]
    blocks = {t.data_ptr() for t in here}
    del here
    got = run(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert not blocks & {t.data_ptr() for t in got}


def test_prefill_host_waits_for_the_stream_that_freed_its_workspace():
    """A workspace that cp_prefill_host makes is a block of the current stream, whose work so
    far comes first."""
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g).bfloat16().pin_memory()  # noqa: E731
    N, KV = sum(NEW), sum(NEW) + sum(PRE)
    o, lse = torch.empty((N, HQ, D), dtype=torch.bfloat16).pin_memory(), torch.empty((N, HQ)).pin_memory()
    batch = (r(N, HQ, D), r(KV, HKV, D), r(KV, HKV, D), o, lse)
    run = lambda **kw: cpa.cp_prefill_host(NEW, PRE, 2, "zigzag", HQ, HKV, D, D, 0.1, [batch],  # noqa: E731
                                           **kw)
    _, streams = run()
    streams[2].synchronize()
    want = o.clone()
    o.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(1 << 29)  # about 0.3 s
    _, streams = run(streams=streams)
    time.sleep(0.05)
    assert not streams[2].query()
    streams[2].synchronize()
    assert torch.equal(o, want)
