"""Attention over shared key runs on the GPU against the fp64 oracle.

Tolerances (u = 2^-8, half a step of bf16; O, L, w_k = softmax weights from the
oracle, `spread` = sum_k w_k |V_k|, `dot` = max_k scale sum_c |q_c K_c|, `smax` =
max |S_k|):
  - a score is an fp32 sum of d exact products and is scaled in base 2, so it is
    off by at most ds = (d + 4) 2^-24 dot + 2^-22 smax;
  - exp and log are off by a few 2^-22, an fp32 sum of n terms by n 2^-24 at
    most, so |dL| <= ds + 2^-19 + n 2^-24 + 2^-22 |L|;
  - every weight is relatively off by at most u (rounded to bf16 for the second
    product) + 2 ds + 2^-19 + n 2^-23, and O moves by that times `spread`; a bf16 O is
    rounded once more, by u |O| (and by 2^-133 where it is subnormal).
"""

import numpy as np
import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L
from oracle import attention as oatt
from oracle import shared as osh

from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


def check(o, lse, ref, d, n_keys, what=""):
    o, lse, out_u = f64(o), f64(lse), U if o.dtype == torch.bfloat16 else 2.0 ** -23
    held = ~np.isnan(ref["lse"])
    emp = np.isneginf(ref["lse"])
    assert (np.isneginf(lse) == emp)[held].all(), what
    assert (o[emp] == 0).all(), what
    fin = held & ~emp
    ds = (d + 4) * 2.0 ** -24 * ref["dot"][fin] + 2.0 ** -22 * ref["smax"][fin]
    tol = ds + 2.0 ** -19 + n_keys * 2.0 ** -24 + 2.0 ** -22 * np.abs(ref["lse"][fin])
    dl = np.abs(lse[fin] - ref["lse"][fin])
    assert (dl <= tol).all(), f"{what}: LSE off by {(dl / tol).max():.2f} of its tolerance"
    rel = U + 2 * ds + 2.0 ** -19 + n_keys * 2.0 ** -23
    tol = rel[:, None] * ref["spread"][fin] + out_u * np.abs(ref["o"][fin]) + 2.0 ** -133
    do = np.abs(o[fin] - ref["o"][fin])
    assert (do <= tol).all(), f"{what}: O off by {(do / tol).max():.2f} of its tolerance"


def make(seed, N, rows, Hq, Hkv, d, quant, std=1.0):
    """q, k, v (device) with the cache's scales, and k, v as fp64 values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q = (r(N, Hq, d) * std).bfloat16()
    k, v = r(rows, Hkv, d).bfloat16(), r(rows, Hkv, d).bfloat16()
    if not quant:
        return q, k, v, {}, f64(k), f64(v)
    cache = cpa.alloc_kv_cache(rows, Hkv, d, d)
    cpa.cp_kv_quantize(cache, k, v)
    kd, vd = cpa.cp_kv_dequantize(cache, out_fp32=True)
    return q, cache.k, cache.v, dict(k_scale=cache.k_scale, v_scale=cache.v_scale), f64(kd), f64(vd)


CASES = {
    # name: Hq, Hkv, d, q_lens, own_lens, prefix
    "one": (8, 2, 128, [1], [1], 0),
    "one_prefix": (32, 8, 128, [1], [1], 1),
    "no_own": (8, 2, 128, [1, 1, 1], [0, 0, 0], 130),
    "nothing": (8, 2, 128, [1, 2], [0, 0], 0),
    "some_nothing": (8, 2, 64, [1, 3, 1], [0, 2, 5], 0),
    "decode": (32, 8, 128, [1] * 7, [1, 127, 128, 129, 300, 0, 64], 517),
    "tile_edges": (4, 4, 128, [1, 1, 1, 1], [255, 256, 257, 1], 256),
    "verify": (8, 2, 128, [3, 1, 8, 5], [3, 40, 200, 5], 385),
    "empty_requests": (8, 2, 64, [0, 2, 0, 1], [50, 20, 0, 0], 77),
    "g3": (12, 4, 128, [1, 2, 4], [9, 130, 4], 333),
    "g5_d64": (40, 8, 64, [1] * 5, [17, 1, 99, 256, 31], 1000),
    "g7": (7, 1, 128, [5, 1], [200, 3], 129),
    "mqa_two_tiles": (32, 1, 128, [2, 9, 1], [31, 9, 400], 640),      # 384 packed rows
    "dual_full": (16, 2, 128, [1] * 32, [5] * 32, 900),               # 256 packed rows
    "dual_ragged": (16, 2, 64, [1] * 19, list(range(19)), 400),       # 152 packed rows
    "many_tiles": (8, 8, 64, [300], [300], 260),                      # causal, 300 packed rows
    "chunk": (8, 4, 128, [150, 70], [400, 70], 140),                  # a prefill chunk
    "long": (8, 2, 128, [1, 1], [3000, 17], 6000),
}


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_oracle(name, quant):
    Hq, Hkv, d, q_lens, own, prefix = CASES[name]
    N, used = sum(q_lens), prefix + sum(own)
    rows = max(1, used) + 3
    q, k, v, scales, k64, v64 = make(len(name), N, rows, Hq, Hkv, d, quant, 1.5)
    scale = d ** -0.5
    segs = cpa.shared_segments(q_lens, own, prefix)
    ref = osh.shared_attention(f64(q), k64, v64, segs.tolist(), scale)
    for ctas, out_t in ((None, torch.bfloat16), (5, torch.float32)):
        plan = cpa.make_shared_plan(q_lens, own, prefix, Hq, Hkv, num_ctas=ctas)
        og, lg = Guarded((N, Hq, d), out_t, 9.0), Guarded((N, Hq), torch.float32, 9.0)
        ws = Guarded((cpa.cp_shared_workspace_size(plan, d),), torch.uint8)
        status = cpa.new_status()
        cpa.cp_attn_shared(plan, q, k, v, scale, **scales, out=og.t, lse=lg.t, workspace=ws.t,
                           status=status)
        cpa.check_status(status, name)
        for x, w in ((og, "O"), (lg, "LSE"), (ws, "workspace")):
            x.check(f"{name} {w}")
        check(og.t, lg.t, ref, d, prefix + max(own), f"{name} ctas={ctas}")


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_outside_the_runs_hold_anything(d, quant):
    """Stale NaN and infinities behind each request's keys, before the prefix and
    between the runs do not reach the outputs; rows past the buffer's end are not
    read (the last run ends inside a tile at the buffer's last row)."""
    Hq, Hkv = 8, 2
    q_lens, own, prefix = [1, 2, 1], [5, 130, 63], 200
    own_row0 = [300, 320, 600]
    rows = 663
    q, k, v, scales, k64, v64 = make(3, 4, rows, Hq, Hkv, d, quant)
    plan = cpa.make_shared_plan(q_lens, own, prefix, Hq, Hkv, prefix_row0=7, own_row0=own_row0)
    live = torch.zeros(rows, dtype=torch.bool)
    live[7:207] = True
    for r0, n in zip(own_row0, own):
        live[r0:r0 + n] = True
    dead = (~live).cuda().nonzero()[:, 0]
    ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), 0.1)
    for t in (k, v):
        if quant:
            t.view(torch.uint8)[dead] = 0x7F  # NaN
        else:
            t[dead] = float("nan")
            t[dead[::2]] = float("inf")
    for s in scales.values():
        s[:, dead] = float("nan")
    o, lse, _ = cpa.cp_attn_shared(plan, q, k, v, 0.1, **scales)
    check(o, lse, ref, d, 330)


@pytest.mark.parametrize("d", [64, 128])
def test_scales_of_many_sizes(d):
    """Cache rows whose scales differ by up to 2^15 lose nothing in the products, in
    units of every kind (4 to 256 packed rows)."""
    Hq, Hkv = 8, 2
    q_lens, own, prefix = [1, 3, 9, 30, 70], [50, 300, 129, 31, 190], 500
    N, rows = sum(q_lens), 1200
    g = torch.Generator(device="cuda").manual_seed(d)
    q = torch.randn(N, Hq, d, generator=g, device="cuda").bfloat16()
    cache = cpa.alloc_kv_cache(rows, Hkv, d, d)
    x = [torch.randn(rows, Hkv, d, generator=g, device="cuda") *
         torch.exp2(torch.randint(-12, 2, (rows, Hkv, 1), generator=g, device="cuda").float())
         for _ in range(2)]
    cpa.cp_kv_quantize(cache, *x)
    for s in (cache.k_scale, cache.v_scale):
        assert 2.0 ** 13 <= (s.max() / s.min()).item() <= 2.0 ** 15
    kd, vd = cpa.cp_kv_dequantize(cache, out_fp32=True)
    plan = cpa.make_shared_plan(q_lens, own, prefix, Hq, Hkv)
    ref = osh.shared_attention(f64(q), f64(kd), f64(vd), plan.segs_host.tolist(), 0.3)
    o, lse, _ = cpa.cp_attn_shared(plan, q, cache.k, cache.v, 0.3, k_scale=cache.k_scale,
                                   v_scale=cache.v_scale, out_fp32=True)
    check(o, lse, ref, d, prefix + max(own))


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("tokens", [1, 9, 64])
def test_many_small_weights(tokens, quant):
    """One key has most of the weight and a value of zero; the others' weights, 2^-18.4
    of it each, make the output (an f16 weight would be subnormal there).  One block to
    a KV head, so that the run is not cut."""
    Hq, Hkv, d, keys = 8, 2, 128, 20000
    q = torch.ones(tokens, Hq, d, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(keys, Hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    k[77], v[77] = 1.0, 0.0
    kw, k64, v64 = {}, f64(k), f64(v)
    if quant:
        cache = cpa.alloc_kv_cache(keys, Hkv, d, d)
        cpa.cp_kv_quantize(cache, k, v)
        k, v, kw = cache.k, cache.v, dict(k_scale=cache.k_scale, v_scale=cache.v_scale)
    scale = 18.4 * np.log(2.0) / d
    plan = cpa.make_shared_plan([1] * tokens, [0] * tokens, keys, Hq, Hkv, num_ctas=2)
    ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), scale)
    o, lse, _ = cpa.cp_attn_shared(plan, q, k, v, scale, **kw, out_fp32=True)
    check(o, lse, ref, d, keys)


def test_nan_in_a_visible_key_reaches_its_rows_only():
    """A NaN among one request's own keys spoils that request and no other."""
    for quant in (False, True):
        q, k, v, scales, k64, v64 = make(4, 3, 500, 8, 2, 128, quant)
        plan = cpa.make_shared_plan([1, 1, 1], [40, 50, 60], 300, 8, 2)
        ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), 0.1)
        if quant:
            k.view(torch.uint8)[350] = 0x7F
        else:
            k[350] = float("nan")
        o, lse, _ = cpa.cp_attn_shared(plan, q, k, v, 0.1, **scales)
        assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
        for key in ref:
            ref[key] = ref[key][[0, 2]]
        check(o[[0, 2]], lse[[0, 2]], ref, 128, 360)


def test_rows_of_no_segment_and_nested_prefixes():
    """Two levels of shared keys over parts of the batch; rows of no segment keep
    what the outputs held."""
    Hq, Hkv, d, N = 8, 2, 128, 12
    q, k, v, _, k64, v64 = make(5, N, 1000, Hq, Hkv, d, False)
    segs = [[1, 9, 199, 0, 0, 200, 0, -1],      # a system prompt
            [1, 4, 149, 0, 200, 150, 0, -1],    # a document of four of the requests
            [6, 3, 9, 0, 400, 10, 0, -1],
            [1, 1, 30, 1, 500, 31, 0, 0], [2, 2, 77, 1, 540, 79, 0, 1], [9, 1, -1, 1, 0, 0, 0, 2],
            [11, 1, 0, 1, 999, 1, 0, 3]]
    plan = cpa.make_shared_plan_segs(segs, N, Hq, Hkv)
    ref = osh.shared_attention(f64(q), k64, v64, segs, 0.09)
    out = torch.full((N, Hq, d), 4.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, Hq), 4.0, device="cuda")
    cpa.cp_attn_shared(plan, q, k, v, 0.09, out=out, lse=lse)
    check(out, lse, ref, d, 430)
    assert (out[[0, 10]] == 4.0).all() and (lse[[0, 10]] == 4.0).all()


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_strides(quant):
    """q from a fused projection, K and V interleaved in one buffer."""
    Hq, Hkv, d, N, rows = 8, 2, 64, 5, 300
    q, k, v, scales, k64, v64 = make(6, N, rows, Hq, Hkv, d, quant)
    fused = torch.randn(N, Hq + 3, d, device="cuda").bfloat16()
    fused[:, 1:1 + Hq] = q
    u8 = (lambda t: t.view(torch.uint8)) if quant else (lambda t: t)
    both = torch.zeros((rows, Hkv, 2, d), dtype=u8(k).dtype, device="cuda")
    both[:, :, 0], both[:, :, 1] = u8(k), u8(v)
    both = both.view(k.dtype)
    if quant:
        wide = torch.zeros((2, Hkv, rows + 10), device="cuda")
        wide[0, :, :rows], wide[1, :, :rows] = scales["k_scale"], scales["v_scale"]
        scales = dict(k_scale=wide[0, :, :rows], v_scale=wide[1, :, :rows])
    plan = cpa.make_shared_plan([1, 3, 1], [20, 30, 40], 210, Hq, Hkv)
    ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), 0.125)
    o, lse, _ = cpa.cp_attn_shared(plan, fused[:, 1:1 + Hq], both[:, :, 0], both[:, :, 1], 0.125,
                                   **scales)
    check(o, lse, ref, d, 250)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_growing_scores(quant):
    """Scores that rise along the keys move the running maximum in every tile;
    large scores make the softmax one-hot."""
    Hq, Hkv, d = 8, 2, 128
    rows = 1500
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn((2, Hq, d), generator=g, device="cuda").abs().bfloat16()
    ramp = torch.linspace(-4, 4, rows, device="cuda")[:, None, None]
    k = (ramp + 0.1 * torch.randn((rows, Hkv, d), generator=g, device="cuda")).bfloat16()
    v = torch.randn((rows, Hkv, d), generator=g, device="cuda").bfloat16()
    scales, k64, v64 = {}, f64(k), f64(v)
    if quant:
        c = cpa.alloc_kv_cache(rows, Hkv, d, d)
        cpa.cp_kv_quantize(c, k, v)
        k64, v64 = (f64(t) for t in cpa.cp_kv_dequantize(c, out_fp32=True))
        k, v, scales = c.k, c.v, dict(k_scale=c.k_scale, v_scale=c.v_scale)
    plan = cpa.make_shared_plan([1, 1], [200, 300], 1000, Hq, Hkv, num_ctas=4)
    for scale in (0.02, 1.0):
        ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), scale)
        o, lse, _ = cpa.cp_attn_shared(plan, q, k, v, scale, out_fp32=True, **scales)
        check(o, lse, ref, d, 1300, f"scale {scale}")


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_same_bits_again_captured_and_on_other_streams(quant):
    q, k, v, scales, k64, v64 = make(9, 20, 3000, 8, 2, 128, quant)
    plan = cpa.make_shared_plan([1] * 20, [5 * i for i in range(20)], 2000, 8, 2)
    run = lambda ws, **kw: cpa.cp_attn_shared(plan, q, k, v, 0.1, workspace=ws, **scales,  # noqa: E731
                                              **kw)
    w1, w2 = (cpa.alloc_shared_workspace(plan, 128) for _ in range(2))
    o, lse, _ = run(w1)
    ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), 0.1)
    check(o, lse, ref, 128, 2100)
    # two calls at once on two streams, each with its workspace
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [run(w1, stream=s1)[:2], run(w2, stream=s2)[:2], run(w1, stream=s1)[:2]]
    torch.cuda.synchronize()
    for oo, ll in outs:
        assert torch.equal(oo, o) and torch.equal(ll, lse)
    # captured: two calls that share a workspace, replayed on new inputs
    og, lg = torch.zeros_like(o), torch.zeros_like(lse)
    oh, lh = torch.zeros_like(o), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(w1, out=og, lse=lg)
        run(w1, out=oh, lse=lh)
    q.copy_(torch.randn_like(q))
    w1.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), 0.1)
    check(og, lg, ref, 128, 2100)
    assert torch.equal(og, oh) and torch.equal(lg, lh)


def test_cache_beyond_two_giga_elements():
    """Key rows whose offsets pass 32 bits."""
    Hkv, d = 8, 128
    rows = (1 << 31) // (Hkv * d) + 1000
    for quant in (False, True):
        q, kt, vt, scales, k64, v64 = make(10, 2, 900, 16, Hkv, d, quant)
        u8 = (lambda t: t.view(torch.uint8)) if quant else (lambda t: t)
        k = torch.empty((rows, Hkv, d), dtype=u8(kt).dtype, device="cuda")
        v = torch.empty_like(k)
        k[-900:], v[-900:] = u8(kt), u8(vt)
        if quant:
            wide = {n: torch.empty((Hkv, rows), device="cuda") for n in scales}
            for n in scales:
                wide[n][:, -900:] = scales[n]
            scales = wide
        plan = cpa.make_shared_plan([1, 1], [100, 300], 500, 16, Hkv, prefix_row0=rows - 900)
        near = cpa.make_shared_plan([1, 1], [100, 300], 500, 16, Hkv)
        ref = osh.shared_attention(f64(q), k64, v64, near.segs_host.tolist(), 0.1)
        o, lse, _ = cpa.cp_attn_shared(plan, q, k.view(kt.dtype), v.view(vt.dtype), 0.1, **scales)
        check(o, lse, ref, d, 800)
        del k, v


def test_table_that_does_not_match_is_reported():
    """Entries that point outside the buffers are skipped and reported; nothing
    outside the outputs is written."""
    q, k, v, _, _, _ = make(11, 4, 600, 8, 2, 128, False)
    plan = cpa.make_shared_plan([1] * 4, [10, 20, 30, 40], 300, 8, 2)
    i = plan.info
    pieces = 8 * i.num_ctas
    units = pieces + 12 * i.num_pieces
    entries = (units + 4 * i.num_units + i.num_q_rows + 2) // 2 * 2
    for at, value in ((pieces + 0, 4), (pieces + 4, 257), (pieces + 4, 200), (pieces + 5, 2),
                      (pieces + 6, 590), (pieces + 6, -1), (pieces + 8, 0),
                      (pieces + 9, int(i.ws_rows)), (6, i.num_pieces + 1), (5, -1), (1, 1),
                      (units + 1, 1 << 30), (units + 2, 257), (units, -1),
                      (entries, i.num_units), (entries + 1, -1)):
        table = plan.table.clone()
        table[at] = value
        bad = cpa.SharedPlan(i, table, plan.segs_host)
        og, lg = Guarded((4, 8, 128), torch.bfloat16), Guarded((4, 8), torch.float32)
        ws = Guarded((cpa.cp_shared_workspace_size(plan, 128),), torch.uint8, 0)
        status = cpa.new_status()
        cpa.cp_attn_shared(bad, q, k, v, 0.1, out=og.t, lse=lg.t, workspace=ws.t, status=status)
        for x in (og, lg, ws):
            x.check(f"word {at}")
        assert int(status.item()) == L.ERR_RANGE, (at, value)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("tokens", [1, 8, 64])
def test_a_wait_that_runs_out_is_reported(tokens, quant):
    """With the queries never published, the waits on them run out in units of every
    kind: the kernel reports it and drains its copies, and the same call is right
    afterwards."""
    lib = L.load()
    Hq, Hkv, d = 8, 2, 128
    q, k, v, scales, k64, v64 = make(9, tokens, 3000, Hq, Hkv, d, quant)
    plan = cpa.make_shared_plan([1] * tokens, [0] * tokens, 3000, Hq, Hkv, num_ctas=7)
    status = cpa.new_status()
    call = lambda: cpa.cp_attn_shared(plan, q, k, v, 0.1, status=status, **scales)  # noqa: E731
    assert lib.cp_attn_debug(L.DEBUG_WAIT_LIMIT_NS, 20_000_000) == L.OK
    assert lib.cp_attn_debug(L.DEBUG_WITHHOLD_Q, 1) == L.OK
    try:
        call()
        torch.cuda.synchronize()
        assert int(status.item()) == L.ERR_TIMEOUT
    finally:
        lib.cp_attn_debug(L.DEBUG_WITHHOLD_Q, 0)
        lib.cp_attn_debug(L.DEBUG_WAIT_LIMIT_NS, 4_000_000_000)
    status.zero_()
    o, lse, _ = call()
    cpa.check_status(status, "after the timeout")
    ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), 0.1)
    check(o, lse, ref, d, 3000)


def test_refusals_of_the_binding():
    q, k, v, scales, _, _ = make(12, 2, 300, 8, 2, 128, True)
    plan = cpa.make_shared_plan([1, 1], [10, 20], 200, 8, 2)
    kb = torch.zeros((300, 2, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        cpa.cp_attn_shared(plan, q, k, v, 0.1, k_scale=scales["k_scale"])
    with pytest.raises(TypeError):
        cpa.cp_attn_shared(plan, q, k, v, 0.1)
    with pytest.raises(TypeError):
        cpa.cp_attn_shared(plan, q, kb, kb, 0.1, **scales)
    with pytest.raises(ValueError):
        cpa.cp_attn_shared(plan, q[:1], kb, kb, 0.1)
    with pytest.raises(ValueError):
        cpa.cp_attn_shared(plan, q, kb, kb[:299], 0.1)
    with pytest.raises(ValueError):
        cpa.cp_attn_shared(plan, q, kb[:, :, :64], kb, 0.1)
    with pytest.raises(L.CpAttnError):
        cpa.cp_attn_shared(plan, q, kb[:229], kb[:229], 0.1)  # the runs reach row 230
    with pytest.raises(L.CpAttnError):
        cpa.cp_attn_shared(plan, q, kb, kb, 0.1, workspace=torch.empty(16, dtype=torch.uint8,
                                                                       device="cuda"))
    with pytest.raises(ValueError):
        cpa.cp_attn_shared(plan, q, k, v, 0.1, k_scale=scales["k_scale"][:, :299],
                           v_scale=scales["v_scale"])


def test_cache_step_decode_and_prefill_together():
    """A serving step end to end: a prompt's K and V go into the quantised cache as
    they are made, a batch of decode queries attends to them behind the shared
    prompt, and the cached prompt is read back as the gathered KV of a prefill."""
    Hq, Hkv, d, P, B = 8, 2, 128, 390, 6
    g = torch.Generator(device="cuda").manual_seed(13)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    cap = 16
    cache = cpa.alloc_kv_cache(P + B * cap, Hkv, d, d)
    kp, vp = r(P, Hkv, d), r(P, Hkv, d)
    cpa.cp_kv_quantize(cache, kp, vp, torch.arange(P, dtype=torch.int32, device="cuda"))
    own0 = [P + b * cap for b in range(B)]
    codes = lambda x: (lambda c, s: c * s.T[:, :, None])(*osh.kv_quantize(f64(x)))  # noqa: E731
    k64, v64 = np.zeros((P + B * cap, Hkv, d)), np.zeros((P + B * cap, Hkv, d))
    k64[:P], v64[:P] = codes(kp), codes(vp)
    for step in range(3):
        kn, vn, q = r(B, Hkv, d), r(B, Hkv, d), r(B, Hq, d)
        slots = [r0 + step for r0 in own0]
        cpa.cp_kv_quantize(cache, kn, vn, torch.tensor(slots, dtype=torch.int32, device="cuda"))
        k64[slots], v64[slots] = codes(kn), codes(vn)
        plan = cpa.make_shared_plan([1] * B, [step + 1] * B, P, Hq, Hkv, own_row0=own0)
        o, lse, _ = cpa.cp_attn_shared(plan, q, cache.k, cache.v, d ** -0.5,
                                       k_scale=cache.k_scale, v_scale=cache.v_scale)
        ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), d ** -0.5)
        check(o, lse, ref, d, P + 3, f"step {step}")
    # request 2 goes on with a prefill of 50 new tokens behind its cached keys
    idx = torch.tensor(list(range(P)) + [own0[2] + i for i in range(3)] + [-1] * 50,
                       dtype=torch.int32, device="cuda")
    kg, vg, q = r(P + 53, Hkv, d), r(P + 53, Hkv, d), r(50, Hq, d)
    new_k, new_v = f64(kg)[-50:], f64(vg)[-50:]
    cpa.cp_kv_dequantize(cache, idx, out_k=kg, out_v=vg)
    prefill = cpa.make_plan([50], [P + 3], 2, "zigzag")
    o, lse = cpa.cp_prefill_attention(q, kg, vg, prefill, d ** -0.5, fuse_restore=True)
    rows = list(range(P)) + [own0[2] + i for i in range(3)]
    O_ref, L_ref = oatt.dense_causal_attention(f64(q), np.concatenate([k64[rows], new_k]),
                                               np.concatenate([v64[rows], new_v]), [50], [P + 3],
                                               d ** -0.5)
    assert np.abs(f64(o) - O_ref).max() <= 2e-2
    assert (np.abs(f64(lse) - L_ref) <= 1e-5 * np.maximum(1, np.abs(L_ref))).all()
