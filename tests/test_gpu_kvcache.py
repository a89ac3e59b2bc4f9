"""Quantised KV cache on the GPU against the fp64 oracle: the codes, scales and
values read back are whole-number exact, so every comparison is for equality."""

import numpy as np
import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L
from oracle import shared as osh

from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

NOTHING = 0x5A  # what unwritten code bytes hold


def f64(t):
    return t.detach().double().cpu().numpy()


def guarded_cache(rows, Hkv, d, dv):
    g = [Guarded((rows, Hkv, d), torch.uint8, NOTHING), Guarded((Hkv, rows), torch.float32, 2.0)]
    if dv:
        g += [Guarded((rows, Hkv, dv), torch.uint8, NOTHING), Guarded((Hkv, rows), torch.float32, 2.0)]
    t = [x.t.view(torch.float8_e4m3fn) if x.t.dtype == torch.uint8 else x.t for x in g]
    return cpa.KVCache(*t), g


def expect(cache_codes, cache_scale, x, slots, rows):
    """Cache contents after the write, from the oracle."""
    codes = np.full(tuple(cache_codes.shape), np.nan)
    codes[:] = torch.full((1,), NOTHING, dtype=torch.uint8).view(torch.float8_e4m3fn).double().item()
    scale = np.full(tuple(cache_scale.shape), 2.0)
    new, sc = osh.kv_quantize(f64(x))
    for i, s in enumerate(slots):
        if 0 <= s < rows:
            codes[s], scale[:, s] = new[i], sc[:, i]
    return codes, scale


def draw(seed, n, H, dim, dtype, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, H, dim, generator=g)
    if spread and n:
        x *= torch.exp2(torch.randint(-30, 30, (n, H, 1), generator=g).float())
    return x.to(dtype).cuda()


@pytest.mark.parametrize("n,H,d,dv", [(1, 1, 16, 16), (5, 2, 64, 64), (33, 8, 128, 128), (7, 1, 576, 0),
                                      (129, 3, 96, 48), (4, 2, 1024, 1024), (300, 4, 192, 128),
                                      (2, 1, 272, 528), (0, 2, 64, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_and_read_back(n, H, d, dv, dtype):
    rows = n + 9
    cache, guards = guarded_cache(rows, H, d, dv)
    k, v = draw(n + d, n, H, d, dtype), draw(n + d + 1, n, H, dv, dtype) if dv else None
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(rows, generator=g)[:n].to(torch.int32)
    slots[2::5] = -1
    status = cpa.new_status()
    cpa.cp_kv_quantize(cache, k, v, slots.cuda(), status=status)
    cpa.check_status(status)
    for x in guards:
        x.check("cache")
    for codes, scale, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        if x is None:
            continue
        want, want_s = expect(codes, scale, x, slots.tolist(), rows)
        assert (f64(codes) == want).all() and (f64(scale) == want_s).all()
    # read back: any row any number of times; negative indices leave the output
    idx = torch.cat([slots, slots[:3], torch.tensor([-1, rows - 1], dtype=torch.int32)])
    for out in (torch.bfloat16, torch.float32):
        ko = Guarded((idx.numel(), H, d), out, 7.0)
        vo = Guarded((idx.numel(), H, dv), out, 7.0) if dv else None
        cpa.cp_kv_dequantize(cache, idx.cuda(), out_k=ko.t, out_v=vo.t if dv else None,
                             status=status)
        cpa.check_status(status)
        for gd, codes, scale in ((ko, cache.k, cache.k_scale), (vo, cache.v, cache.v_scale)):
            if gd is None:
                continue
            gd.check("read back")
            val = f64(codes) * f64(scale).T[:, :, None]
            want = val[idx.clamp_min(0).numpy()]
            want[idx.numpy() < 0] = 7.0
            got = f64(gd.t)
            fin = np.isfinite(want)  # the codes of unwritten rows may stand for anything
            assert (got[fin] == want[fin]).all() and (np.isnan(got) == np.isnan(want)).all()


def test_special_values():
    """Zeros, subnormals, the largest values, ties, infinities and NaN; a row's
    infinity or NaN does not change the scale of its other elements."""
    rows = [torch.zeros(64), torch.full((64,), 2.0 ** -133), torch.full((64,), 3.3895e38),
            torch.linspace(-500, 500, 64), torch.arange(64) * 0.0625 + 1.0,
            torch.full((64,), 448.0), torch.full((64,), 449.0), torch.full((64,), 2.0 ** -126),
            torch.linspace(-1, 1, 64), torch.linspace(-1, 1, 64)]
    rows[8][5], rows[8][6] = float("inf"), float("-inf")
    rows[9][7] = float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.stack(rows).to(dtype)[:, None].cuda()
        cache = cpa.alloc_kv_cache(len(rows), 1, 64, 64)
        cpa.cp_kv_quantize(cache, x, x)
        want, want_s = osh.kv_quantize(f64(x))
        for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            got = f64(c)
            assert (np.isnan(got) == np.isnan(want)).all() and (f64(s) == want_s).all()
            assert (got[~np.isnan(want)] == want[~np.isnan(want)]).all()
        k, _ = cpa.cp_kv_dequantize(cache)
        val = want * want_s.T[:, :, None]
        assert np.isfinite(val[:9]).all()
        assert (f64(k)[~np.isnan(val)] == val[~np.isnan(val)]).all()
        assert np.isnan(f64(k)[9, 0, 7]) and np.isnan(f64(k)).sum() == 1


def test_strided_rows_and_cache():
    """k and v as views of a fused projection, the cache as K / V interleaved rows."""
    n, H, d = 37, 4, 64
    fused = draw(3, n, 3 * H, d, torch.bfloat16)
    k, v = fused[:, H:2 * H], fused[:, 2 * H:]
    both = torch.zeros((64, 2, H, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((2, H, 100), device="cuda")
    cache = cpa.KVCache(both[:, 0], scales[0, :, :64], both[:, 1], scales[1, :, :64])
    slots = (torch.arange(n, dtype=torch.int32) + 11).cuda()
    cpa.cp_kv_quantize(cache, k, v, slots)
    for c, s, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        want, want_s = osh.kv_quantize(f64(x))
        assert (f64(c)[11:11 + n] == want).all() and (f64(s)[:, 11:11 + n] == want_s).all()
        assert (f64(c)[:11] == 0).all() and (f64(c)[11 + n:] == 0).all()
    assert (scales[:, :, 64:] == 0).all()


def test_one_row_or_head_of_any_stride():
    """The stride of a dimension of one entry means nothing."""
    x = draw(5, 3, 3, 64, torch.bfloat16).reshape(-1)
    for shape, strides in (((1, 2, 64), (7, 64, 1)), ((3, 1, 64), (64, 3, 1)), ((1, 1, 64), (1, 1, 1))):
        k = torch.as_strided(x, shape, strides)
        cache = cpa.alloc_kv_cache(shape[0], shape[1], 64, 64)
        cpa.cp_kv_quantize(cache, k, k)
        want, want_s = osh.kv_quantize(f64(k))
        assert (f64(cache.k) == want).all() and (f64(cache.v_scale) == want_s).all()


def test_cache_without_rows():
    cache = cpa.alloc_kv_cache(0, 2, 64, 64)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    cpa.cp_kv_quantize(cache, none, none)
    k, v = cpa.cp_kv_dequantize(cache)
    assert k.shape == v.shape == (0, 2, 64)
    status = cpa.new_status()
    one = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    cpa.cp_kv_quantize(cache, one, one, status=status)
    assert int(status.item()) == L.ERR_RANGE
    skip = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    status = cpa.new_status()
    cpa.cp_kv_quantize(cache, one, one, skip, status=status)
    cpa.cp_kv_dequantize(cache, skip, out_k=one, out_v=one.clone(), status=status)
    cpa.check_status(status)
    assert (one == 1).all()


def test_index_out_of_range_is_reported_and_skipped():
    cache = cpa.alloc_kv_cache(8, 2, 64, 64)
    x = draw(1, 3, 2, 64, torch.bfloat16)
    status = cpa.new_status()
    cpa.cp_kv_quantize(cache, x, x, torch.tensor([1, 8, 2], dtype=torch.int32, device="cuda"),
                       status=status)
    assert int(status.item()) == L.ERR_RANGE
    want, _ = osh.kv_quantize(f64(x))
    assert (f64(cache.k)[[1, 2]] == want[[0, 2]]).all()
    assert (f64(cache.k)[[0, 3, 4, 5, 6, 7]] == 0).all()
    # more rows than the cache has, without slots
    status.zero_()
    cpa.cp_kv_quantize(cache, draw(1, 9, 2, 64, torch.bfloat16), draw(2, 9, 2, 64, torch.bfloat16),
                       status=status)
    assert int(status.item()) == L.ERR_RANGE
    status.zero_()
    out = torch.full((2, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    cpa.cp_kv_dequantize(cache, torch.tensor([8, 1], dtype=torch.int32, device="cuda"), out_k=out,
                         status=status)
    assert int(status.item()) == L.ERR_RANGE and (out[0] == 5.0).all()
    assert (f64(out)[1] == f64(cache.k)[1] * f64(cache.k_scale)[:, 1][:, None]).all()


def test_refusals_of_the_binding():
    cache = cpa.alloc_kv_cache(8, 2, 64, 64)
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        cpa.cp_kv_quantize(cache, x.half(), x.half())
    with pytest.raises(TypeError):
        cpa.cp_kv_quantize(cache, x, x.float())
    with pytest.raises(ValueError):
        cpa.cp_kv_quantize(cache, x)
    with pytest.raises(ValueError):
        cpa.cp_kv_quantize(cache, x, x[:1])
    with pytest.raises(ValueError):
        cpa.cp_kv_quantize(cache, x[:, :, :32], x)
    with pytest.raises(ValueError):
        cpa.cp_kv_quantize(cache, x.transpose(1, 2), x)
    with pytest.raises(TypeError):
        cpa.cp_kv_quantize(cache, x, x, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        cpa.cp_kv_quantize(cache, x, x, torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        cpa.cp_kv_dequantize(cache, out_k=x)
    with pytest.raises(TypeError):
        cpa.cp_kv_dequantize(cpa.KVCache(cache.k.view(torch.uint8), cache.k_scale))
    with pytest.raises(ValueError):
        cpa.cp_kv_quantize(cpa.KVCache(cache.k, cache.k_scale.t().contiguous().t()), x)
    cpa.cp_kv_quantize(cache, x[:0], x[:0])  # no rows: nothing to do


def test_captured_and_replayed_on_another_stream():
    cache = cpa.alloc_kv_cache(40, 2, 128, 128)
    k, v = draw(1, 20, 2, 128, torch.bfloat16), draw(2, 20, 2, 128, torch.bfloat16)
    slots = torch.arange(20, dtype=torch.int32, device="cuda")
    idx = torch.arange(40, dtype=torch.int32, device="cuda")
    ko = torch.zeros((40, 2, 128), dtype=torch.bfloat16, device="cuda")
    vo = torch.zeros_like(ko)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cpa.cp_kv_quantize(cache, k, v, slots)
        cpa.cp_kv_dequantize(cache, idx, out_k=ko, out_v=vo)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa.cp_kv_quantize(cache, k, v, slots)
        cpa.cp_kv_dequantize(cache, idx, out_k=ko, out_v=vo)
    k.copy_(draw(7, 20, 2, 128, torch.bfloat16))
    v.copy_(draw(8, 20, 2, 128, torch.bfloat16))
    slots.add_(13)
    graph.replay()
    torch.cuda.synchronize()
    for x, out in ((k, ko), (v, vo)):
        want, sc = osh.kv_quantize(f64(x))
        assert (f64(out)[13:33] == want * sc.T[:, :, None]).all()


def test_cache_beyond_two_giga_elements():
    """Rows whose code offsets pass 32 bits."""
    H, d = 8, 128
    rows = (1 << 31) // (H * d) + 4096
    codes = torch.empty((rows, H, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cache = cpa.KVCache(codes, torch.empty((H, rows), device="cuda"))
    x = draw(5, 64, H, d, torch.bfloat16)
    slots = torch.arange(rows - 64, rows, dtype=torch.int32, device="cuda")
    cpa.cp_kv_quantize(cache, x, slots=slots)
    out, _ = cpa.cp_kv_dequantize(cache, slots)
    want, sc = osh.kv_quantize(f64(x))
    assert (f64(out) == want * sc.T[:, :, None]).all()
