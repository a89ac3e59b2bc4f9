"""Attention over shared key runs where the score factor of the e4m3 path leaves fp32's
normal range.  That path multiplies raw scores of a tile by scale * 2^(e_k - f), with
2^f max|q| of the row in [2^14, 2^15) and e_k the tile's largest scale exponent.

Tolerances are those of test_gpu_shared.py."""

import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from oracle import shared as osh

from test_gpu_shared import check, f64

pytestmark = pytest.mark.gpu

# query tokens that make units of up to 8, of 9 to 128 and of more than 128 packed rows
KINDS = pytest.mark.parametrize("tokens", [1, 9, 64], ids=["small", "single", "dual"])
CACHES = pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
DIMS = pytest.mark.parametrize("d", [64, 128])


def attend(q, k, v, quant, tokens, own, prefix, scale, what):
    """The call on k, v (quantised first) against the oracle: a prefix that ends inside a
    KV tile, and the tokens' own causal keys."""
    Hq, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    kw, k64, v64 = {}, f64(k), f64(v)
    if quant:
        cache = cpa.alloc_kv_cache(k.shape[0], Hkv, d, d)
        cpa.cp_kv_quantize(cache, k, v)
        k64, v64 = (f64(t) for t in cpa.cp_kv_dequantize(cache, out_fp32=True))
        k, v, kw = cache.k, cache.v, dict(k_scale=cache.k_scale, v_scale=cache.v_scale)
    for ctas in (2, None):
        plan = cpa.make_shared_plan([tokens], [own], prefix, Hq, Hkv, num_ctas=ctas)
        ref = osh.shared_attention(f64(q), k64, v64, plan.segs_host.tolist(), scale)
        o, lse, _ = cpa.cp_attn_shared(plan, q, k, v, scale, **kw, out_fp32=True)
        check(o, lse, ref, d, prefix + own, f"{what}, {ctas} blocks")


def draw(seed, tokens, rows, d, Hq=8, Hkv=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return r(tokens, Hq, d), r(rows, Hkv, d), r(rows, Hkv, d)


@KINDS
@CACHES
@DIMS
def test_zero_queries_and_zero_keys(d, quant, tokens):
    """The masked keys of a tile stay out of a row whose factor is below fp32's range:
    zero queries over zero keys give the mean of V and L = ln n, zero values 0."""
    prefix, scale = 300, d ** -0.5
    for own in (tokens + 37, max(1, tokens // 2)):  # (the latter: rows that see none of them)
        q, k, v = draw(own, tokens, prefix + own, d)
        zq, zk = torch.zeros_like(q), torch.zeros_like(k)
        attend(zq, zk, v, quant, tokens, own, prefix, scale, "zero queries and keys")
        attend(zq, zk, torch.zeros_like(v), quant, tokens, own, prefix, scale, "all zero")
        one = q.clone()
        one[tokens // 2] = 0
        attend(one, (k.float() * 2.0 ** -20).bfloat16(), v, quant, tokens, own, prefix, scale,
               "one zero query, keys of 2^-20")
        some = k.clone()
        some[128:256] = 0
        some[prefix:] = 0
        attend((q.float() * 2.0 ** -20).bfloat16(), some, v, quant, tokens, own, prefix, scale,
               "queries of 2^-20, a tile of zero keys")


@KINDS
@CACHES
@DIMS
def test_large_queries_orthogonal_to_large_keys(d, quant, tokens):
    """Scores of 0 between queries of 2^100 and keys of 2^60, whose factor is above
    fp32's range: the mean of V and L = ln n."""
    prefix, own = 300, tokens + 37
    q, k, v = draw(d, tokens, prefix + own, d)
    q[:, :, : d // 2] = 0
    k[:, :, d // 2:] = 0
    attend((q.float() * 2.0 ** 100).bfloat16(), (k.float() * 2.0 ** 60).bfloat16(), v, quant,
           tokens, own, prefix, d ** -0.5, "orthogonal")
