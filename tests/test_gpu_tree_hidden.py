"""New keys in an e4m3 cache that a row does not see may have any scale: 2^100 of the others', an
infinity or NaN.  Tolerances are those of test_gpu_shared."""

import numpy as np
import pytest
import torch

from oracle import paged as op

from test_gpu_shared import check, make
from test_gpu_tree import Step, i32

pytestmark = pytest.mark.gpu

# heads and nodes: units of 8, 16, 128 and 256 packed rows, and new keys over several tiles
UNITS = {"8": (4, 2, 4), "16": (8, 2, 4), "single": (8, 2, 20), "dual": (8, 2, 64), "tiles": (4, 2, 300),
         "small_tiles": (2, 2, 300)}
SCALES = pytest.mark.parametrize("value", [2.0 ** 100, 2.0 ** 30, float("inf"), float("nan")], ids=str)


def step(name, seed, cached=(150, 0, 41)):
    """A batch whose requests' masks hide two keys: node 1 from every row, node 2 from all but
    the rows 2 and the last."""
    Hq, Hkv, nodes = UNITS[name]
    s = Step(seed, [nodes] * len(cached), list(cached), 16, tree=False)
    seen = []
    for n in s.nodes:
        see = np.tril(np.ones((n, n), dtype=bool))
        see[:, 1] = False
        see[:, 2] = False
        see[[2, n - 1], 2] = True
        seen.append(see)
    words = -(-nodes // 32)
    bits = np.zeros((s.N, 32 * words), dtype=np.uint64)
    bits[:, :nodes] = np.concatenate(seen)
    packed = (bits.reshape(s.N, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    kw = dict(mask=i32(packed.view(np.int32).tolist()).view(s.N, words), max_nodes=1 if name == "small_tiles" else nodes)
    first = np.array(s.q_start[:-1])
    return s, Hq, Hkv, seen, kw, first


@SCALES
@pytest.mark.parametrize("side", ["k_scale", "v_scale"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", sorted(UNITS))
def test_scales_of_keys_that_rows_do_not_see(name, d, side, value):
    s, Hq, Hkv, seen, kw, first = step(name, 31)
    q, k, v, scales, k64, v64 = make(31, s.N, s.rows, Hq, Hkv, d, True)
    at = np.array(s.slots)
    hidden, part = at[first + 1], at[first + 2]
    big = scales[side].clone()
    big[:, i32(hidden.tolist()).long()] = value
    big[:, i32(part.tolist()).long()] = value
    x64 = k64 if side == "k_scale" else v64
    x64[hidden] = 0.0  # (of no row's sums)
    x64[part] *= np.nan_to_num(value, nan=0.0, posinf=0.0) / scales[side][:, part].t().cpu().numpy()[..., None]
    sees = np.concatenate([first + 2, first + s.nodes[0] - 1])
    rest = np.setdiff1d(np.arange(s.N), sees)
    ref = s.ref(q, k64, v64, 0.05, seen)
    for ctas in (None, 3):
        o, lse, _ = s.call(q, k, v, 0.05, num_ctas=ctas, out_fp32=True, **{**scales, side: big}, **kw)
        check(o[rest], lse[rest], {n: x[rest] for n, x in ref.items()}, d, 460, "rows that do not see it")
        if side == "v_scale" and np.isfinite(value):
            check(o[sees], lse[sees], {n: x[sees] for n, x in ref.items()}, d, 460, "rows that see it")
        elif side == "v_scale":
            assert torch.isnan(o[sees]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", sorted(UNITS))
def test_a_hidden_key_changes_no_bit(name, d):
    """The rows that do not see a key have the same bits whatever its scale and codes are."""
    s, Hq, Hkv, _, kw, first = step(name, 32)
    q, k, v, scales, _, _ = make(32, s.N, s.rows, Hq, Hkv, d, True)
    want = s.call(q, k, v, 0.05, **scales, **kw)
    at = i32(np.array(s.slots)[first + 1].tolist()).long()
    for value, code in ((2.0 ** 110, 0x7E), (2.0 ** -117, 0x00), (float("nan"), 0x7F)):
        k2, v2 = k.clone(), v.clone()
        k2.view(torch.uint8)[at], v2.view(torch.uint8)[at] = code, code
        s2 = {n: x.clone() for n, x in scales.items()}
        for x in s2.values():
            x[:, at] = value
        o, lse, _ = s.call(q, k2, v2, 0.05, **s2, **kw)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("tokens", [4, 20, 64])
def test_a_chains_later_tokens(tokens):
    """Without a mask a chain's last token has a scale that the rows before it must not feel."""
    Hq, Hkv, d = 8, 2, 128
    s = Step(33, [tokens, tokens], [100, 230], 16, tree=False)
    q, k, v, scales, k64, v64 = make(33, s.N, s.rows, Hq, Hkv, d, True)
    last = [s.slots[tokens - 1], s.slots[-1]]
    ref = s.ref(q, k64, v64, 0.1)
    rows = [i for i in range(s.N) if i % tokens != tokens - 1]
    for name in scales:
        big = scales[name].clone()
        big[:, i32(last).long()] = 2.0 ** 90
        o, lse, _ = s.call(q, k, v, 0.1, **{**scales, name: big})
        check(o[rows], lse[rows], {n: x[rows] for n, x in ref.items()}, d, 300, name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", sorted(UNITS))
def test_new_values_of_many_sizes(name, d):
    """New and cached values whose scales step up and down by up to 2^15: what O is taken
    relative to moves in either direction between tiles of cached and of new keys."""
    for up in (12, -12):
        s, Hq, Hkv, seen, kw, _ = step(name, 34, (150, 300, 41))
        q, k, v, scales, k64, v64 = make(34, s.N, s.rows, Hq, Hkv, d, True)
        f = torch.ones(s.rows)
        f[s.slots] = 2.0 ** up
        f[s.slots[::5]] = 2.0 ** (up // 2)
        scales["v_scale"] *= f.cuda()
        v64 *= f.double().numpy()[:, None, None]
        ref = s.ref(q, k64, v64, 0.05, seen)
        for ctas in (None, 2):
            o, lse, _ = s.call(q, k, v, 0.05, num_ctas=ctas, out_fp32=True, **scales, **kw)
            check(o, lse, ref, d, 600, f"2^{up}")


def test_the_oracle_leaves_a_hidden_key_out():
    see = np.eye(2, dtype=bool)
    q, k, v = np.ones((2, 1, 4)), np.ones((16, 1, 4)), np.arange(16.0)[:, None, None] * np.ones((1, 1, 4))
    k[1], v[1] = 1e30, 1e30
    got = op.tree_attention(q, k, v, [0, 2], [0], [[0]], 16, [see], 0.1)
    assert got["o"][0, 0, 0] == 0.0
