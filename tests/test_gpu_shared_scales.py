"""The e4m3 path of attention over shared key runs at its own tolerance (weights in f16),
with scales that move along the run and that lie far below the largest."""

import numpy as np
import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from oracle import shared as osh

from test_gpu_shared import f64
from test_gpu_shared_edges import DIMS, KINDS, draw

pytestmark = pytest.mark.gpu


def check_f16(o, lse, ref, d, n_keys, q, k64, v64, scale, lost, what):
    """The e4m3 path against the oracle, its terms alone (o and lse fp32).  An element of K
    or V that is not exact in f16 is off by at most `lost` of the largest element of its
    tile (or run), a query element by at most 2^-39 of the row's largest:
        ds = (d + 4) 2^-24 dot + 2^-22 smax + scale sum|q| max|K| (lost + 2^-39).
    A weight is off by at most 2^-11 of itself and 2^-32 of the largest (P in f16), and by
    2 ds + 2^-19 + n 2^-23 of itself as in check(); O moves by that times spread, and for
    the absolute part by 2^-32 n max|V|, and by lost max|V|; O's own rounding is 2^-23 |O|."""
    o, lse = f64(o), f64(lse)
    emp = np.isneginf(ref["lse"])
    assert (np.isneginf(lse) == emp).all() and (o[emp] == 0).all(), what
    fin = ~emp
    wide = np.abs(f64(q)).sum(-1)[fin] * scale * np.abs(k64).max()
    ds = (d + 4) * 2.0 ** -24 * ref["dot"][fin] + 2.0 ** -22 * ref["smax"][fin] + \
        wide * (lost + 2.0 ** -39)
    tol = ds + 2.0 ** -19 + n_keys * 2.0 ** -24 + 2.0 ** -22 * np.abs(ref["lse"][fin])
    dl = np.abs(lse[fin] - ref["lse"][fin])
    assert (dl <= tol).all(), f"{what}: LSE off by {(dl / tol).max():.2f} of its tolerance"
    rel = 2.0 ** -11 + 2 * ds + 2.0 ** -19 + n_keys * 2.0 ** -23
    top = np.abs(v64).max()
    tol = rel[:, None] * ref["spread"][fin] + 2.0 ** -23 * np.abs(ref["o"][fin]) + \
        (2.0 ** -32 * n_keys + lost) * top
    do = np.abs(o[fin] - ref["o"][fin])
    assert (do <= tol).all(), f"{what}: O off by {(do / tol).max():.2f} of its tolerance"


def cached(k, v):
    """The quantised cache of rows k, v, and what it stands for in 64 bits."""
    cache = cpa.alloc_kv_cache(k.shape[0], k.shape[1], k.shape[2], v.shape[2])
    cpa.cp_kv_quantize(cache, k, v)
    return (cache, *(f64(t) for t in cpa.cp_kv_dequantize(cache, out_fp32=True)))


@KINDS
@DIMS
@pytest.mark.parametrize("below", [14, 15, 18, 22, 24, 25, 30])
def test_scales_far_below_the_largest(below, d, tokens):
    """Rows 2^-below under the largest scale: down to 2^-24 an element is off by at most
    2^-32 of the largest element, below that the row may count as zeros (2^-24)."""
    lost = 2.0 ** -32 if below <= 24 else 2.0 ** -24
    keys, Hq, Hkv = 300, 8, 2
    g = torch.Generator(device="cuda").manual_seed(below)
    u = lambda: 225 + 223 * torch.rand((keys, Hkv, d), generator=g, device="cuda")  # noqa: E731
    small = (torch.arange(keys, device="cuda") % 3 == 1)[:, None, None]
    plan = cpa.make_shared_plan([1] * tokens, [0] * tokens, keys, Hq, Hkv, num_ctas=2)
    run = lambda c, q, scale: cpa.cp_attn_shared(plan, q, c.k, c.v, scale, k_scale=c.k_scale,  # noqa: E731
                                                 v_scale=c.v_scale, out_fp32=True)[:2]
    segs = plan.segs_host.tolist()
    # K: the large rows see nothing of q, the small ones' scores are 0.5 to 1
    lower = torch.arange(d, device="cuda") < d // 2
    q = torch.where(lower, 0.0, torch.ones((tokens, Hq, d), device="cuda")).bfloat16()
    k = torch.where(small, torch.where(lower, 0.0, u() * 2.0 ** -below), torch.where(lower, u(), 0.0))
    cache, k64, v64 = cached(k, u())
    assert cache.k_scale.max().item() == 2.0 ** below * cache.k_scale.min().item()
    scale = 2.0 ** below / (448 * (d // 2))
    ref = osh.shared_attention(f64(q), k64, v64, segs, scale)
    check_f16(*run(cache, q, scale), ref, d, keys, q, k64, v64, scale, lost, "K")
    # V: one small row has nearly all of the weight
    k = torch.zeros((keys, Hkv, d), device="cuda")
    k[100] = 1.0
    q = torch.ones((tokens, Hq, d), device="cuda").bfloat16()
    assert small[100]
    cache, k64, v64 = cached(k, torch.where(small, u() * 2.0 ** -below, u()))
    scale = 60.0 / d
    ref = osh.shared_attention(f64(q), k64, v64, segs, scale)
    check_f16(*run(cache, q, scale), ref, d, keys, q, k64, v64, scale, lost, "V")


@KINDS
@DIMS
@pytest.mark.parametrize("ctas", [2, 6])
@pytest.mark.parametrize("steps", [(3,), (-3,), (5, -4), (0, 7, 0, -6), (1, 1, 1, -8)], ids=str)
def test_values_whose_scales_step_along_the_run(steps, ctas, d, tokens):
    """V of a KV tile is 2^steps[t] times the tile's before it, so that the exponent of O moves
    inside a piece (2 blocks: about 9 tiles a piece and several pieces a stream), and starts
    again with the next.  Uniform weights: what any tile adds, and a missing or wrong
    rescale of it, is far above f16's 2^-11 of a weight."""
    Hq, Hkv, prefix = 16, 4, 8 * 128 + 61
    own = tokens + 300
    rows = prefix + own
    q, k, v = draw(sum(steps) + d, tokens, rows, d, Hq, Hkv)
    e, exps = 0, []
    for t in range(-(-rows // 128)):
        exps.append(e)
        e += steps[t % len(steps)]
    # (within 2^12 of the run's largest, where f16 loses nothing)
    x = torch.tensor(exps, device="cuda").float()
    x = torch.maximum(x, x.max() - 12).repeat_interleave(128)[:rows]
    v = v.float() * torch.exp2(x)[:, None, None]
    cache, k64, v64 = cached(k.float(), v)
    plan = cpa.make_shared_plan([tokens], [own], prefix, Hq, Hkv, num_ctas=ctas)
    scale = 0.02
    ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), scale)
    o, lse, _ = cpa.cp_attn_shared(plan, q, cache.k, cache.v, scale, k_scale=cache.k_scale,
                                   v_scale=cache.v_scale, out_fp32=True)
    check_f16(o, lse, ref, d, rows, q, k64, v64, scale, 2.0 ** -32, f"{steps}")


@KINDS
@DIMS
def test_weights_of_the_e4m3_path_in_f16(d, tokens):
    """Ordinary values at f16's own tolerance, in the order of the oracle's terms."""
    own, prefix = tokens + 200, 1500
    q, k, v = draw(d + 1, tokens, prefix + own, d)
    cache, k64, v64 = cached(k, v)
    for ctas in (2, None):
        plan = cpa.make_shared_plan([tokens], [own], prefix, 8, 2, num_ctas=ctas)
        ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), d ** -0.5)
        o, lse, _ = cpa.cp_attn_shared(plan, q, cache.k, cache.v, d ** -0.5, k_scale=cache.k_scale,
                                       v_scale=cache.v_scale, out_fp32=True)
        check_f16(o, lse, ref, d, prefix + own, q, k64, v64, d ** -0.5, 2.0 ** -32, f"{ctas} blocks")
