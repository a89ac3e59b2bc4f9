"""fp64 oracle of rotary positions, of the layout of a decode step over a paged cache, and of
the attention of its new rows.

Key j of request b lies at cache row table[b][j // page] * page + j % page; request b has
kv_lens[b] cached keys, and its new rows q_start[b] .. q_start[b+1]-1 follow as keys.
"""

from decimal import Decimal, getcontext

import numpy as np

from . import shared as osh

TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021")


def angles(positions, inv_freq, axis):
    """positions[axis_c][row] * inv_freq_c mod 2 pi, [n, pairs]; a far position's product
    does not fit 64 bits, so it is taken in 50 digits."""
    getcontext().prec = 60
    positions, inv_freq = np.asarray(positions), np.asarray(inv_freq, dtype=np.float64)
    at = positions[np.asarray(axis)].T.astype(np.int64)  # [n, pairs]
    out = at * inv_freq
    for i, c in zip(*np.nonzero(np.abs(at) >= 1 << 20)):
        out[i, c] = float(Decimal(int(at[i, c])) * Decimal(float(inv_freq[c])) % TWO_PI)
    return out


def rotate(x, positions, inv_freq, axis=None, first=0, interleaved=False, inverse=False):
    """The rows x [n, heads, d] with their pairs turned; positions [axes, n]."""
    y = np.array(x, dtype=np.float64)
    pairs = len(inv_freq)
    t = angles(positions, inv_freq, np.zeros(pairs, int) if axis is None else axis)[:, None]
    c, s = np.cos(t), np.sin(t) * (-1 if inverse else 1)
    at = np.arange(pairs)
    i, j = (first + 2 * at, first + 2 * at + 1) if interleaved else (first + at, first + pairs + at)
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def tree_layout(q_start, kv_lens, table, page, parents, num_rows):
    """(slots, positions, ancestors as a bool matrix a request) of a step's new rows."""
    slots, positions, seen = [-1] * num_rows, [0] * num_rows, []
    for b, n in enumerate(kv_lens):
        T = q_start[b + 1] - q_start[b]
        see = np.zeros((T, T), dtype=bool)
        for i in range(T):
            row = q_start[b] + i
            slots[row] = table[b][(n + i) // page] * page + (n + i) % page
            up = i - 1 if parents is None else parents[row]
            see[i] = see[up] if up >= 0 else False
            see[i, i] = True
            positions[row] = n + int(see[i].sum()) - 1
        seen.append(see)
    return slots, positions, seen


def mask_words(seen, words):
    """The bool matrices of tree_layout as int32 words, all requests' rows in order."""
    rows = sum(len(s) for s in seen)
    out, at = np.zeros((rows, words), dtype=np.uint32), 0
    for s in seen:
        for i, j in zip(*np.nonzero(s)):
            out[at + i, j // 32] |= np.uint32(1 << (j % 32))
        at += len(s)
    return out.view(np.int32)


def tree_attention(q, k, v, q_start, kv_lens, table, page, seen, scale):
    """As oracle.shared.shared_attention, for new rows over a paged cache; seen[b] [T, T]:
    which of the request's new keys each of its rows sees."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    N, Hq, _ = q.shape
    dv = v.shape[2]
    out = dict(o=np.full((N, Hq, dv), np.nan), lse=np.full((N, Hq), np.nan),
               spread=np.zeros((N, Hq, dv)), smax=np.zeros((N, Hq)), dot=np.zeros((N, Hq)))
    for b, n in enumerate(kv_lens):
        T = q_start[b + 1] - q_start[b]
        keys = np.arange(n + T)
        rows = np.asarray(table[b], dtype=np.int64)[keys // page] * page + keys % page if n + T else keys
        for i in range(T):
            at = rows[np.concatenate([np.ones(n, dtype=bool), seen[b][i]])]
            row = q_start[b] + i
            one = osh.shared_attention(q[row:row + 1], k[at], v[at], [(0, 1, len(at) - 1, 0, 0)], scale)
            for name in out:
                out[name][row] = one[name][0]
    return out
