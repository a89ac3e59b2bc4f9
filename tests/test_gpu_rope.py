"""Rotary positions, alone and on the way into a cache, against the fp64 oracle.

Tolerances of a rotated pair (a, b), for fp32 arithmetic of unit 2^-24:
  - the phase is cut at 2^-32 turns and the rest of a quarter turn (at most pi/4) is
    rounded once, so the angle is off by less than 2^-29 + 2^-24; cos and sin themselves by
    at most 2 units in the last place, 2^-23: together below 2^-22;
  - each product and the sum round once: 2^-24 (|a| + |b|) each.
So a result is off by less than 2^-21 (|a| + |b|) before it is rounded to its type: bf16
2^-8 of its size, fp32 2^-24.
"""

import numpy as np
import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L
from oracle import paged as op
from oracle import shared as osh

from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().double().cpu().numpy()


def freqs(pairs, base=10000.0):
    return base ** (-np.arange(pairs) / pairs)


def size(x, rot):
    """|a| + |b| of each element's pair."""
    pairs, first, inter = rot["pairs"], rot["first"], rot["interleaved"]
    s = np.abs(f64(x))
    at = np.arange(pairs)
    i, j = (first + 2 * at, first + 2 * at + 1) if inter else (first + at, first + pairs + at)
    both = s[..., i] + s[..., j]
    s[..., i] = s[..., j] = both
    return s


def draw(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * 2).to(dtype).cuda()


def make(seed, n, pairs, axes=1, first=0, interleaved=False, far=4096):
    g = torch.Generator().manual_seed(seed)
    axis = torch.randint(0, axes, (pairs,), generator=g)
    axis[-1] = axes - 1
    pos = torch.randint(-far, far, (axes, n), generator=g).to(torch.int32)
    rot = dict(pairs=pairs, first=first, interleaved=interleaved)
    rope = cpa.make_rope(freqs(pairs), axes=axis, first=first, interleaved=interleaved)
    return rope, pos.cuda(), rot, dict(positions=pos.numpy(), inv_freq=freqs(pairs), axis=axis.numpy(),
                                       first=first, interleaved=interleaved)


def check(got, x, rot, ref, what=""):
    got, step = f64(got), STEP[got.dtype]
    tol = 2.0 ** -21 * size(x, rot) + step * np.abs(ref) * (1 + 2.0 ** -20) + 2.0 ** -133
    assert (np.abs(got - ref) <= tol).all(), f"{what}: {(np.abs(got - ref) / tol).max():.2f} of the tolerance"


SHAPES = {
    # n, Hq, Hk, d, pairs, axes, first
    "one": (1, 1, 0, 16, 8, 1, 0),
    "head": (3, 4, 2, 128, 64, 1, 0),
    "axes": (37, 5, 3, 128, 64, 3, 0),
    "part": (130, 8, 1, 96, 16, 2, 0),
    "latent": (33, 2, 1, 576, 32, 1, 512),
    "middle": (9, 3, 2, 80, 24, 1, 16),
    "wide": (2, 2, 2, 1024, 512, 8, 0),
    "wider": (5, 1, 1, 528, 8, 1, 8),
    "batch": (2500, 7, 1, 64, 32, 1, 0),
}


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_rotation(name, dtype, interleaved):
    n, Hq, Hk, d, pairs, axes, first = SHAPES[name]
    rope, pos, rot, ref = make(n + d, n, pairs, axes, first, interleaved)
    q, k = draw(1, (n, Hq, d), dtype), draw(2, (n, Hk, d), dtype) if Hk else None
    for inverse in (False, True):
        oq, ok = Guarded((n, Hq, d), dtype), Guarded((n, max(Hk, 1), d), dtype)
        status = cpa.new_status()
        cpa.cp_rope(rope, q, k, pos, inverse=inverse, out_q=oq.t, out_k=ok.t if Hk else None, status=status)
        cpa.check_status(status)
        for x, o, name in ((q, oq, "q"), (k, ok, "k")):
            o.check(name)
            if x is not None:
                check(o.t, x, rot, op.rotate(f64(x), **ref, inverse=inverse), name)


def test_far_positions():
    """Positions up to 32 bits, of either sign, with frequencies above a turn."""
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 987654321, -123456789, 1 << 20]],
                       dtype=torch.int32)
    f = np.concatenate([[1.0, np.pi, 100.0, -3.7, 2.0 ** 20, 1e-9, 0.0], 0.5 ** np.arange(9)])
    rope = cpa.make_rope(f)
    x = draw(3, (9, 2, 32), torch.float32)
    y, _ = cpa.cp_rope(rope, x, None, pos.cuda()[0])
    check(y, x, dict(pairs=16, first=0, interleaved=False), op.rotate(f64(x), pos.numpy(), f))


def test_gradient_is_the_inverse():
    """<g, R x> = <R^T g, x>, against differences of the loss, and R^T R = 1."""
    rope, pos, rot, ref = make(5, 11, 16, 2)
    x, g = draw(4, (11, 3, 64), torch.float32), draw(5, (11, 3, 64), torch.float32)
    back, _ = cpa.cp_rope(rope, g, None, pos, inverse=True)
    check(back, g, rot, op.rotate(f64(g), **ref, inverse=True))
    # the loss <g, R x> is linear: its difference along a direction is exact but for rounding
    e = draw(6, (11, 3, 64), torch.float32)
    loss = lambda t: float((f64(cpa.cp_rope(rope, t, None, pos)[0]) * f64(g)).sum())  # noqa: E731
    up = (x + e)
    diff, want = loss(up) - loss(x), float((f64(back) * (f64(up) - f64(x))).sum())
    room = 2.0 ** -20 * float((np.abs(f64(g)) * (size(up, rot) + size(x, rot) + size(e, rot))).sum())
    assert abs(diff - want) <= room
    again, _ = cpa.cp_rope(rope, cpa.cp_rope(rope, x, None, pos)[0], None, pos, inverse=True)
    assert (np.abs(f64(again) - f64(x)) <= 2.0 ** -19 * size(x, rot)).all()


def test_strides_and_in_place():
    """Views of a fused projection, heads before rows, broadcast inputs, in place."""
    n, Hq, Hk, d = 21, 4, 2, 64
    rope, pos, rot, ref = make(6, n, 32)
    fused = draw(7, (n, Hq + 2 * Hk, d), torch.bfloat16)
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hk]
    before, wq, wk = fused.clone(), op.rotate(f64(q), **ref), op.rotate(f64(k), **ref)
    turned = torch.zeros((Hq, n, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    cpa.cp_rope(rope, q, k, pos, out_q=turned, out_k=fused[:, Hq + Hk:])
    check(turned, q, rot, wq)
    check(fused[:, Hq + Hk:], k, rot, wk)
    assert torch.equal(fused[:, :Hq + Hk], before[:, :Hq + Hk])
    cpa.cp_rope(rope, q, k, pos, out_q=q, out_k=k)
    check(fused[:, :Hq], before[:, :Hq], rot, wq)
    check(fused[:, Hq:Hq + Hk], before[:, Hq:Hq + Hk], rot, wk)
    one = draw(8, (1, 1, d), torch.bfloat16).expand(n, Hq, d)
    y, _ = cpa.cp_rope(rope, one, None, pos)
    check(y, one, rot, op.rotate(f64(one), **ref))


def test_special_values_stay_in_their_pair():
    rope, pos, rot, ref = make(9, 3, 8)
    x = draw(9, (3, 2, 32), torch.float32)
    clean = cpa.cp_rope(rope, x, None, pos)[0]
    x[1, 0, 2], x[2, 1, 20] = float("nan"), float("inf")
    y = cpa.cp_rope(rope, x, None, pos)[0]
    assert torch.isnan(y[1, 0, [2, 10]]).all() and y[2, 1, 20] == float("inf")
    other = torch.ones_like(x, dtype=torch.bool)
    other[1, 0, [2, 10]] = other[2, 1, 20] = False
    assert torch.equal(y[other], clean[other])


def paged(rows, Hkv, d, dv, quant):
    """A cache of guarded buffers full of 2.0 (codes: 0x40), and the buffers."""
    if not quant:
        g = [Guarded((rows, Hkv, d), torch.bfloat16, 2.0)] + \
            ([Guarded((rows, Hkv, dv), torch.bfloat16, 2.0)] if dv else [])
        return (g[0].t, g[1].t if dv else None), g
    g = []
    for dim in (d, dv):
        if dim:
            g += [Guarded((rows, Hkv, dim), torch.uint8, 0x40), Guarded((Hkv, rows), torch.float32, 1.0)]
    return cpa.KVCache(*[x.t.view(torch.float8_e4m3fn) if x.t.dtype == torch.uint8 else x.t for x in g]), g


def check_codes(codes, scales, x, rot, ref, slots):
    """Codes and scales of rotated rows: the scale is that of a maximum within the
    rotation's error of the exact one, the value within half a step."""
    room = 2.0 ** -21 * size(x, rot)
    for i, s in enumerate(slots):
        if s < 0:
            continue
        for h in range(ref.shape[1]):
            a, r = np.abs(ref[i, h]).max(), room[i, h].max()
            sc = scales[h, s].item()
            e = {int(osh.scale_exponents(np.array([m]))) for m in (max(a - r, 0.0), a, a + r)}
            assert np.log2(sc) in e
            off = np.abs(f64(codes[s, h]) * sc - ref[i, h])
            assert (off <= 2.0 ** -4 * np.abs(ref[i, h]) + 2.0 ** -10 * sc + 2 * room[i, h]).all()


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,Hq,Hkv,d,dv,pairs,axes,first", [
    (1, 4, 2, 128, 128, 64, 1, 0), (70, 8, 2, 64, 64, 16, 3, 0), (33, 0, 1, 576, 0, 32, 1, 512),
    (19, 3, 3, 96, 48, 48, 1, 0), (900, 2, 1, 128, 64, 64, 1, 0), (4, 2, 2, 48, 1024, 16, 1, 8)])
def test_append(n, Hq, Hkv, d, dv, pairs, axes, first, dtype, quant):
    rows = n + 11
    for inter in (False, True):
        rope, pos, rot, ref = make(n + d, n, pairs, axes, first, inter)
        q = draw(1, (n, Hq, d), dtype) if Hq else None
        k, v = draw(2, (n, Hkv, d), dtype), draw(3, (n, Hkv, dv), dtype) if dv else None
        cache, guards = paged(rows, Hkv, d, dv, quant)
        slots = torch.randperm(rows, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
        slots[1::4] = -1
        status = cpa.new_status()
        oq = cpa.cp_kv_append(cache, k, v, slots.cuda(), rope=rope, positions=pos, q=q, status=status)
        cpa.check_status(status)
        for g in guards:
            g.check("cache")
        if Hq:
            check(oq, q, rot, op.rotate(f64(q), **ref), "q")
        want = op.rotate(f64(k), **ref)
        kept, at = (slots >= 0).numpy(), slots[slots >= 0].long()
        rest = torch.ones(rows, dtype=torch.bool)
        rest[at] = False
        if quant:
            check_codes(cache.k, cache.k_scale, k, rot, want, slots.tolist())
            if dv:
                codes, sc = osh.kv_quantize(f64(v))
                assert (f64(cache.v)[at] == codes[kept]).all() and (f64(cache.v_scale)[:, at] == sc[:, kept]).all()
            assert (cache.k.view(torch.uint8)[rest.cuda()] == 0x40).all()
            assert (cache.k_scale[:, rest.cuda()] == 1.0).all()
        else:
            check(cache[0][at.cuda()], k[torch.tensor(kept).cuda()], rot, want[kept], "k")
            assert (cache[0][rest.cuda()] == 2.0).all()
            if dv:
                assert torch.equal(cache[1][at.cuda()], v[torch.tensor(kept).cuda()].bfloat16())
                assert (cache[1][rest.cuda()] == 2.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_without_rotation_is_the_quantised_write(dtype):
    n, H, d, dv = 50, 3, 64, 128
    k, v = draw(1, (n, H, d), dtype), draw(2, (n, H, dv), dtype)
    k[3, 1, 5], k[4, 0, 7], v[5] = float("inf"), float("nan"), 0.0
    a, b = cpa.alloc_kv_cache(60, H, d, dv), cpa.alloc_kv_cache(60, H, d, dv)
    slots = torch.arange(n, dtype=torch.int32, device="cuda").flip(0) + 3
    assert cpa.cp_kv_append(a, k, v, slots) is None
    cpa.cp_kv_quantize(b, k, v, slots)
    for x, y in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)
    # without slots row i goes to cache row i
    cpa.cp_kv_append(a, k, v)
    cpa.cp_kv_quantize(b, k, v)
    assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8))


def test_slots_and_axes_outside_are_reported():
    rope, pos, _, _ = make(1, 4, 16)
    k = draw(1, (4, 2, 64), torch.bfloat16)
    (ck, cv), guards = paged(10, 2, 64, 64, False)
    status = cpa.new_status()
    slots = torch.tensor([3, 10, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    cpa.cp_kv_append((ck, cv), k, k, slots, rope=rope, positions=pos, status=status)
    for g in guards:
        g.check("cache")
    assert int(status.item()) == L.ERR_RANGE
    kept = torch.ones(10, dtype=torch.bool)
    kept[3] = False
    assert (ck[kept.cuda()] == 2.0).all() and (ck[3] != 2.0).any()
    # more rows than the cache has, without slots
    status.zero_()
    cpa.cp_kv_append((ck[:2], cv[:2]), k, k, rope=rope, positions=pos, status=status)
    for g in guards:
        g.check("cache")
    assert int(status.item()) == L.ERR_RANGE and (cv[4:] == 2.0).all()
    # a pair whose axis has no row of positions
    status.zero_()
    bad = cpa.make_rope(freqs(16), axes=[1] * 16)
    bad = cpa.Rope(bad.table, axes=1)
    y, _ = cpa.cp_rope(bad, k, None, pos, status=status)
    assert int(status.item()) == L.ERR_RANGE and torch.equal(y, k)


def test_captured_and_on_another_stream():
    rope, pos, rot, ref = make(2, 40, 32)
    q, k = draw(1, (40, 4, 64), torch.bfloat16), draw(2, (40, 2, 64), torch.bfloat16)
    cache, _ = paged(64, 2, 64, 64, True)
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    oq = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    cpa.cp_kv_append(cache, k, k, slots, rope=rope, positions=pos, q=q, out_q=oq)
    with torch.cuda.graph(graph):
        cpa.cp_kv_append(cache, k, k, slots, rope=rope, positions=pos, q=q, out_q=oq)
    q.copy_(draw(3, q.shape, torch.bfloat16))
    pos.add_(17)
    slots.copy_(slots.flip(0) + 20)
    graph.replay()
    torch.cuda.synchronize()
    ref["positions"] = pos.cpu().numpy()
    check(oq, q, rot, op.rotate(f64(q), **ref))
    check_codes(cache.k, cache.k_scale, k, rot, op.rotate(f64(k), **ref), slots.tolist())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, z = cpa.cp_rope(rope, q, k, pos, stream=side)
    side.synchronize()
    assert torch.equal(y, oq)
    check(z, k, rot, op.rotate(f64(k), **ref))


def test_rows_beyond_two_giga_elements():
    """A cache whose offsets pass 32 bits, in elements and bytes."""
    Hkv, d = 8, 128
    rows = (1 << 31) // (Hkv * d) + 50
    rope, pos, rot, ref = make(4, 3, 64)
    k = draw(1, (3, Hkv, d), torch.bfloat16)
    ck = torch.empty((rows, Hkv, d), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([rows - 1, 5, rows - 30], dtype=torch.int32, device="cuda")
    cpa.cp_kv_append((ck, None), k, None, slots, rope=rope, positions=pos)
    check(ck[slots.long()], k, rot, op.rotate(f64(k), **ref))
