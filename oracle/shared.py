"""fp64 oracle of the quantised KV cache and of attention over shared key runs.

Quantisation of one vector x: a = max finite |x_c|, e = clamp(ceil(log2(a/448)),
-117, 119), code = e4m3(x / 2^e) (nearest even, saturated), value = code 2^e.

Shared attention: query row n sees, for every segment that holds it (row i of the
segment), the run's keys 0 .. q_pos0 + i*q_pos_step; softmax over all of them.
"""

import numpy as np


def scale_exponents(x):
    """e of every vector (last axis) of x."""
    a = np.abs(np.where(np.isfinite(x), x, 0.0)).max(-1)
    m, e = np.frexp(a)  # a = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = e - 9 + (m > 0.875)
    return np.clip(np.where(a > 0, e, -117), -117, 119).astype(np.int64)


def e4m3(y):
    """y rounded to the nearest e4m3 value (ties to even), saturated at 448."""
    y = np.asarray(y, dtype=np.float64)
    c = np.clip(y, -448.0, 448.0)
    _, e = np.frexp(np.abs(np.where(np.isfinite(c), c, 0.0)))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.round(c / step) * step


def kv_quantize(x):
    """(code values, scales) of the rows x [n, Hkv, dim]: codes like x, scales [Hkv, n]."""
    x = np.asarray(x, dtype=np.float64)
    e = scale_exponents(x)
    return e4m3(x / np.exp2(e.astype(np.float64))[..., None]), np.exp2(e.astype(np.float64)).T


def row_runs(segs, num_q_rows):
    """For each query row the list of (first KV row, visible keys) of its segments."""
    runs = [[] for _ in range(num_q_rows)]
    for s in segs:
        q_row0, q_len, q_pos0, step, kv_row0 = (int(v) for v in s[:5])
        for i in range(q_len):
            runs[q_row0 + i].append((kv_row0, max(0, q_pos0 + i * step + 1)))
    return runs


def shared_attention(q, k, v, segs, scale):
    """Returns dict(o, lse, spread, smax, dot): O [N, Hq, dv], L [N, Hq]; spread =
    sum_k w_k |V_k| (how far a relative error of the weights can move O), smax =
    max |S_k| and dot = max_k scale * sum_c |q_c K_c| (what rounding of the scores
    is relative to).  Rows of no segment: NaN."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    N, Hq, _ = q.shape
    Hkv, dv = v.shape[1], v.shape[2]
    g = Hq // Hkv
    o = np.full((N, Hq, dv), np.nan)
    spread = np.zeros((N, Hq, dv))
    lse = np.full((N, Hq), np.nan)
    smax, dot = np.zeros((N, Hq)), np.zeros((N, Hq))
    for n, runs in enumerate(row_runs(segs, N)):
        if not runs:
            continue
        at = np.concatenate([np.arange(r0, r0 + c) for r0, c in runs]).astype(np.int64)
        if at.size == 0:
            o[n], lse[n] = 0.0, -np.inf
            continue
        for h in range(Hkv):
            kk, vv, qq = k[at, h], v[at, h], q[n, h * g:(h + 1) * g]
            s = scale * (qq @ kk.T)
            m = s.max(-1, keepdims=True)
            w = np.exp(s - m)
            tot = w.sum(-1, keepdims=True)
            hs = slice(h * g, (h + 1) * g)
            lse[n, hs] = (m + np.log(tot))[:, 0]
            o[n, hs] = w @ vv / tot
            spread[n, hs] = w @ np.abs(vv) / tot
            smax[n, hs] = np.abs(s).max(-1)
            dot[n, hs] = scale * (np.abs(qq) @ np.abs(kk).T).max(-1)
    return dict(o=o, lse=lse, spread=spread, smax=smax, dot=dot)
