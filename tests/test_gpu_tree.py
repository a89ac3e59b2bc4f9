"""Decode steps over a paged cache on the GPU: their layout, equal to the oracle's, and the
attention of their new rows against the fp64 oracle, with the tolerances of the shared-key
attention (the same arithmetic: see test_gpu_shared)."""

import random

import numpy as np
import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L
from oracle import paged as op
from oracle import shared as osh

from test_gpu_guards import Guarded
from test_gpu_shared import check, f64, make

pytestmark = pytest.mark.gpu

KINDS = pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """A batch over a paged cache whose pages lie in any order, with trees of its nodes."""

    def __init__(self, seed, nodes, kv, page, spare=2, tree=True, width=None):
        rng = random.Random(seed)
        self.nodes, self.kv, self.page, self.N = nodes, kv, page, sum(nodes)
        need = [-(-(n + k) // page) for n, k in zip(nodes, kv)]
        self.rows = (sum(need) + spare) * page
        free = list(range(self.rows // page))
        rng.shuffle(free)
        width = max([1] + need) if width is None else width
        self.table = [[free.pop() for _ in range(n)] + [-1] * (width - n) for n in need]
        self.q_start = [sum(nodes[:b]) for b in range(len(nodes) + 1)]
        self.parents = [rng.randint(max(-1, i - 5), i - 1) for n in nodes for i in range(n)] if tree else None
        self.dev = dict(page_table=i32(self.table), q_start=i32(self.q_start), kv_lens=i32(kv))
        self.slots, self.positions, self.seen = op.tree_layout(self.q_start, kv, self.table, page, self.parents,
                                                               self.N)
        self.words = max(1, -(-max([1] + nodes) // 32))
        self.mask = i32(op.mask_words(self.seen, self.words).tolist()).view(self.N, self.words) if tree else None

    def ref(self, q, k64, v64, scale, seen=None):
        return op.tree_attention(f64(q), k64, v64, self.q_start, self.kv, self.table, self.page,
                                 self.seen if seen is None else seen, scale)

    def call(self, q, k, v, scale, **kw):
        kw = {"mask": self.mask, "max_nodes": max([1] + self.nodes), **kw}
        return cpa.cp_attn_tree(q, k, v, self.dev["page_table"], self.page, self.dev["q_start"],
                                self.dev["kv_lens"], scale, **kw)


LAYOUTS = {
    "one": ([1], [0], 16), "chain": ([9], [30], 16), "some": ([3, 0, 70, 1, 33], [5, 100, 0, 16, 47], 32),
    "long": ([2500, 64], [7, 130], 64), "many": ([1 + b % 5 for b in range(300)], [3 * b for b in range(300)], 128),
}


@pytest.mark.parametrize("tree", [True, False], ids=["tree", "chain"])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_layout(name, tree):
    s = Step(len(name), *LAYOUTS[name], tree=tree)
    pad = 5
    N = s.N + pad
    parents = i32(s.parents + [-7] * pad) if tree else None
    outs = [Guarded((N,), torch.int32), Guarded((N,), torch.int32), Guarded((N, s.words), torch.int32)]
    status = cpa.new_status()
    got = cpa.cp_tree_layout(s.dev["q_start"], s.dev["kv_lens"], s.dev["page_table"], s.page, N, parents=parents,
                             slots=outs[0].t, positions=outs[1].t, mask=outs[2].t if tree else None, status=status)
    cpa.check_status(status)
    for g in outs:
        g.check(name)
    assert got[0].tolist() == s.slots + [-1] * pad and got[1].tolist() == s.positions + [0] * pad
    if tree:
        assert torch.equal(got[2][: s.N], s.mask) and (got[2][s.N:] == 0).all()
    made = cpa.cp_tree_layout(s.dev["q_start"], s.dev["kv_lens"], s.dev["page_table"], s.page, s.N,
                              parents=parents, max_nodes=max(s.nodes))
    assert torch.equal(made[0], got[0][: s.N]) and (made[2] is None or torch.equal(made[2], s.mask))


def test_layout_reports_what_does_not_fit():
    s = Step(1, [4, 3], [20, 30], 16)
    base = dict(s.dev, parents=i32(s.parents))

    def run(words=1, **kw):
        a = {**base, **kw}
        status = cpa.new_status()
        outs = [Guarded((7,), torch.int32, 55), Guarded((7,), torch.int32, 55), Guarded((7, words), torch.int32, 55)]
        cpa.cp_tree_layout(a["q_start"], a["kv_lens"], a["page_table"], 16, 7, parents=a["parents"], slots=outs[0].t,
                           positions=outs[1].t, mask=outs[2].t, status=status)
        for g in outs:
            g.check(str(kw))
        return int(status.item()), outs[0].t.tolist(), outs[2].t[:, 0].tolist()

    assert run()[0] == L.OK
    table = s.dev["page_table"].clone()
    table[0, 1] = -1
    code, slots, _ = run(page_table=table)
    assert code == L.ERR_RANGE and slots == [-1] * 4 + s.slots[4:]
    for kw in (dict(kv_lens=i32([-1, 30])), dict(kv_lens=i32([1000, 30])), dict(kv_lens=i32([2 ** 31 - 2, 30]))):
        code, slots, _ = run(**kw)
        assert code == L.ERR_RANGE and slots == [-1] * 4 + s.slots[4:], kw
    for kw in (dict(q_start=i32([0, 9, 7])), dict(q_start=i32([0, -4, 7])), dict(q_start=i32([1, 4, 7])),
               dict(q_start=i32([0, 4, 2 ** 31 - 1]))):
        assert run(**kw)[0] == L.ERR_RANGE, kw
    # a parent that is not below its node counts as none
    for up in (2, 3, -2, 2 ** 31 - 1, -2 ** 31):
        code, _, mask = run(parents=i32([-1, 0, up, 2, -1, 0, 1]))
        assert code == L.ERR_RANGE and mask == [1, 3, 4, 12, 1, 3, 7], up


CASES = {
    # name: Hq, Hkv, d, nodes, cached keys, page
    "one": (8, 2, 128, [1], [0], 16),
    "one_more": (32, 8, 128, [1], [1], 16),
    "decode": (32, 8, 128, [1] * 7, [1, 127, 128, 129, 300, 0, 64], 16),
    "padded": (8, 2, 64, [1, 0, 1, 0], [50, 70, 0, 0], 32),
    "tile_edges": (4, 4, 128, [1] * 5, [126, 127, 128, 255, 511], 128),
    "pages_end_in_tiles": (8, 2, 128, [2, 3, 1], [15, 16, 1000], 64),
    "chain8": (32, 8, 128, [8, 5, 1, 8], [0, 333, 128, 1021], 16),
    "tree26": (16, 2, 64, [26, 13, 20], [77, 0, 640], 32),
    "tree64": (32, 8, 128, [64, 40, 61], [130, 1000, 3], 16),
    "tree_over_tiles": (4, 2, 128, [200, 33], [100, 250], 256),
    "g3": (12, 4, 128, [1, 2, 4], [9, 130, 4], 16),
    "g5_d64": (40, 8, 64, [1, 3, 7, 2], [17, 1, 99, 256], 64),
    "g7": (7, 1, 128, [5, 1], [200, 3], 16),
    "mqa": (32, 1, 128, [2, 9, 1], [31, 9, 400], 32),
    "g64": (64, 1, 64, [1, 3], [700, 20], 16),
    "chunk": (8, 4, 128, [300, 70], [40, 140], 16),
    "long": (8, 2, 128, [1, 4], [3000, 6017], 1024),
    "requests": (2, 1, 64, [b % 3 for b in range(700)], [b % 37 for b in range(700)], 16),
}


@KINDS
@pytest.mark.parametrize("tree", [True, False], ids=["tree", "chain"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_attention(name, tree, quant):
    Hq, Hkv, d, nodes, kv, page = CASES[name]
    s = Step(len(name), nodes, kv, page, tree=tree)
    q, k, v, scales, k64, v64 = make(len(name), s.N + 3, s.rows, Hq, Hkv, d, quant, 1.5)
    scale = d ** -0.5
    ref = s.ref(q[: s.N], k64, v64, scale)
    mask = None if s.mask is None else torch.cat([s.mask, s.mask.new_full((3, s.words), -1)])
    for ctas, out_t, most in ((None, torch.bfloat16, max(nodes)), (5, torch.float32, 1)):
        og, lg = Guarded((s.N + 3, Hq, d), out_t, 9.0), Guarded((s.N + 3, Hq), torch.float32, 9.0)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        ws = Guarded((cpa.cp_tree_workspace_size(Hq, Hkv, d, most, ctas or sms),), torch.uint8, 0xFF)
        status = cpa.new_status()
        s.call(q, k, v, scale, mask=mask, max_nodes=most, num_ctas=ctas, out=og.t, lse=lg.t, workspace=ws.t,
               status=status, **scales)
        cpa.check_status(status, name)
        for x, w in ((og, "O"), (lg, "LSE"), (ws, "workspace")):
            x.check(f"{name} {w}")
        assert (og.t[s.N:] == 9.0).all() and (lg.t[s.N:] == 9.0).all()
        check(og.t[: s.N], lg.t[: s.N], ref, d, max(a + b for a, b in zip(nodes, kv)), f"{name} {ctas}")


@KINDS
@pytest.mark.parametrize("heads", [(4, 2), (16, 2), (16, 1)])
def test_any_mask(heads, quant):
    """Masks of random bits: rows that see nothing, keys that no row sees, bits behind a
    request's last row."""
    Hq, Hkv = heads
    s = Step(3, [33, 1, 64, 7], [0, 0, 130, 260], 16)
    g = torch.Generator().manual_seed(4)
    bits = torch.rand((s.N, 96), generator=g) < 0.2
    bits[[0, 5, 33, 40]] = False
    bits[:, 3] = False
    words = [sum(int(x) << j for j, x in enumerate(row[32 * w: 32 * w + 32])) for row in bits for w in range(3)]
    mask = i32([w - (1 << 32) if w >= 1 << 31 else w for w in words]).view(s.N, 3)
    seen = [bits[a:b, : b - a].numpy() for a, b in zip(s.q_start, s.q_start[1:])]
    q, k, v, scales, k64, v64 = make(5, s.N, s.rows, Hq, Hkv, 128, quant)
    # the keys that no row sees hold anything
    for b, n in enumerate(s.kv):
        for j in range(s.nodes[b]):
            if not seen[b][:, j].any():
                row = s.slots[s.q_start[b] + j]
                for t in (k, v):
                    if quant:
                        t.view(torch.uint8)[row] = 0x7F
                    else:
                        t[row] = float("nan")
    ref = s.ref(q, np.nan_to_num(k64), np.nan_to_num(v64), 0.09, seen)
    assert np.isneginf(ref["lse"][[0, 5, 33]]).all()
    o, lse, _ = s.call(q, k, v, 0.09, mask=mask, **scales)
    check(o, lse, ref, 128, 330)


@KINDS
@pytest.mark.parametrize("nodes", [[1, 3], [8, 6], [30, 64]])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_outside_hold_anything(d, nodes, quant):
    """NaN and infinities in every cache row that no request's keys are in, scales
    among them."""
    s = Step(6, nodes, [150, 41], 64, spare=5)
    q, k, v, scales, k64, v64 = make(6, s.N, s.rows, 8, 2, d, quant)
    live = torch.zeros(s.rows, dtype=torch.bool)
    for b, n in enumerate(s.kv):
        for j in range(n + s.nodes[b]):
            live[s.table[b][j // 64] * 64 + j % 64] = True
    dead = (~live).cuda().nonzero()[:, 0]
    ref = s.ref(q, k64, v64, 0.1)
    for t in (k, v):
        if quant:
            t.view(torch.uint8)[dead] = 0x7F
        else:
            t[dead] = float("nan")
            t[dead[::2]] = float("inf")
    for x in scales.values():
        x[:, dead] = float("nan")
    o, lse, _ = s.call(q, k, v, 0.1, **scales)
    check(o, lse, ref, d, 220)


@KINDS
@pytest.mark.parametrize("heads,nodes", [((2, 2), 7), ((8, 2), 7), ((16, 1), 7), ((32, 1), 7)])
def test_values_that_some_rows_do_not_see(heads, nodes, quant):
    """A new key whose value is NaN or infinite spoils the rows that see it and no other."""
    Hq, Hkv = heads
    s = Step(7, [nodes, 3], [140, 20], 16, tree=False)
    q, k, v, scales, k64, v64 = make(7, s.N, s.rows, Hq, Hkv, 128, quant)
    seen = [np.tril(np.ones((n, n), dtype=bool)) for n in s.nodes]
    seen[0][:, 2] = seen[0][:, 5] = False
    seen[0][[2, 4], 2] = seen[0][5, 5] = True
    mask = i32(op.mask_words(seen, 1).tolist())
    for node, value in ((2, float("inf")), (5, float("nan"))):
        if quant:
            v.view(torch.uint8)[s.slots[node], :, 77] = 0x7F
        else:
            v[s.slots[node], :, 77] = value
    ref = s.ref(q, k64, np.nan_to_num(v64), 0.1, seen)
    o, lse, _ = s.call(q, k, v, 0.1, mask=mask, **scales)
    bad = [2, 4, 5]
    assert torch.isnan(o[bad]).all()
    good = [i for i in range(s.N) if i not in bad]
    check(o[good], lse[good], {n: x[good] for n, x in ref.items()}, 128, 150)


@KINDS
@pytest.mark.parametrize("nodes", [1, 4, 40])
def test_growing_scores(nodes, quant):
    """Scores that rise along the keys move the running maximum in every step; large
    scores make the softmax one-hot."""
    Hq, Hkv, d = 8, 2, 128
    s = Step(8, [nodes, nodes], [1200, 1001], 16)
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn((s.N, Hq, d), generator=g, device="cuda").abs().bfloat16()
    k = torch.zeros((s.rows, Hkv, d), device="cuda")
    for b, n in enumerate(s.kv):
        at = torch.tensor([s.table[b][j // 16] * 16 + j % 16 for j in range(n + nodes)], device="cuda")
        k[at] = torch.linspace(-4, 4, n + nodes, device="cuda")[:, None, None]
    k = (k + 0.1 * torch.randn(k.shape, generator=g, device="cuda")).bfloat16()
    v = torch.randn(k.shape, generator=g, device="cuda").bfloat16()
    scales, k64, v64 = {}, f64(k), f64(v)
    if quant:
        c = cpa.alloc_kv_cache(s.rows, Hkv, d, d)
        cpa.cp_kv_quantize(c, k, v)
        k64, v64 = (f64(t) for t in cpa.cp_kv_dequantize(c, out_fp32=True))
        k, v, scales = c.k, c.v, dict(k_scale=c.k_scale, v_scale=c.v_scale)
    for scale in (0.02, 1.0):
        ref = s.ref(q, k64, v64, scale)
        o, lse, _ = s.call(q, k, v, scale, out_fp32=True, num_ctas=4, **scales)
        check(o, lse, ref, d, 1250, f"scale {scale}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [1, 3, 7, 40])
def test_scales_of_many_sizes(nodes, d):
    """Cache rows whose scales differ by up to 2^15 lose nothing in the products."""
    s = Step(9, [nodes, nodes], [500, 333], 16)
    g = torch.Generator(device="cuda").manual_seed(d)
    q = torch.randn(s.N, 8, d, generator=g, device="cuda").bfloat16()
    cache = cpa.alloc_kv_cache(s.rows, 2, d, d)
    x = [torch.randn(s.rows, 2, d, generator=g, device="cuda") *
         torch.exp2(torch.randint(-12, 2, (s.rows, 2, 1), generator=g, device="cuda").float()) for _ in range(2)]
    cpa.cp_kv_quantize(cache, *x)
    kd, vd = cpa.cp_kv_dequantize(cache, out_fp32=True)
    ref = s.ref(q, f64(kd), f64(vd), 0.3)
    o, lse, _ = s.call(q, cache.k, cache.v, 0.3, k_scale=cache.k_scale, v_scale=cache.v_scale, out_fp32=True)
    check(o, lse, ref, d, 560)


@KINDS
@pytest.mark.parametrize("nodes", [1, 4, 40])
def test_zero_queries_and_keys(nodes, quant):
    """Zero queries over zero keys: the mean of V and L = ln n."""
    s = Step(10, [nodes], [300], 16, tree=False)
    q, k, v, scales, k64, v64 = make(10, s.N, s.rows, 4, 2, 64, quant)
    q.zero_()
    k.view(torch.uint8).zero_() if quant else k.zero_()
    if quant:
        scales["k_scale"].fill_(2.0 ** -117)
    ref = s.ref(q, 0 * k64, v64, 0.125)
    o, lse, _ = s.call(q, k, v, 0.125, **scales)
    check(o, lse, ref, 64, 340)


@KINDS
def test_strides(quant):
    """q from a fused projection, K and V interleaved in one buffer, wide tables."""
    Hq, Hkv, d = 8, 2, 64
    s = Step(11, [1, 9, 4], [20, 130, 40], 32, width=9)
    q, k, v, scales, k64, v64 = make(11, s.N, s.rows, Hq, Hkv, d, quant)
    fused = torch.randn(s.N, Hq + 3, d, device="cuda").bfloat16()
    fused[:, 1:1 + Hq] = q
    u8 = (lambda t: t.view(torch.uint8)) if quant else (lambda t: t)
    both = torch.zeros((s.rows, Hkv, 2, d), dtype=u8(k).dtype, device="cuda")
    both[:, :, 0], both[:, :, 1] = u8(k), u8(v)
    both = both.view(k.dtype)
    if quant:
        wide = torch.zeros((2, Hkv, s.rows + 10), device="cuda")
        wide[0, :, : s.rows], wide[1, :, : s.rows] = scales["k_scale"], scales["v_scale"]
        scales = dict(k_scale=wide[0, :, : s.rows], v_scale=wide[1, :, : s.rows])
    s.dev["page_table"] = s.dev["page_table"].repeat(1, 2)[:, :9]
    ref = s.ref(q, k64, v64, 0.125)
    o, lse, _ = s.call(fused[:, 1:1 + Hq], both[:, :, 0], both[:, :, 1], 0.125, **scales)
    check(o, lse, ref, d, 150)


@KINDS
@pytest.mark.parametrize("nodes", [1, 20])
def test_same_bits_again_captured_and_on_other_streams(nodes, quant):
    """The same call gives the same bits; a captured one replays on other lengths, pages and
    masks of its batch, and two captured graphs take turns on a workspace."""
    s = Step(12, [nodes] * 12, [97 * i for i in range(12)], 16, width=90)
    t = Step(13, [nodes] * 12, [1200 - 90 * i for i in range(12)], 16, width=90)
    rows = max(s.rows, t.rows)
    q, k, v, scales, k64, v64 = make(12, s.N, rows, 8, 2, 128, quant)
    w1, w2 = (cpa.alloc_tree_workspace(8, 2, 128, nodes) for _ in range(2))
    o, lse, _ = s.call(q, k, v, 0.1, workspace=w1, **scales)
    check(o, lse, s.ref(q, k64, v64, 0.1), 128, 1200)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [s.call(q, k, v, 0.1, workspace=w, stream=x, **scales)[:2] for w, x in ((w1, s1), (w2, s2), (w1, s1))]
    torch.cuda.synchronize()
    for oo, ll in outs:
        assert torch.equal(oo, o) and torch.equal(ll, lse)
    og, lg, oh, lh = (torch.zeros_like(x) for x in (o, lse, o, lse))
    graphs = []
    for a, b in ((og, lg), (oh, lh)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.call(q, k, v, 0.1, workspace=w1, out=a, lse=b, **scales)
    for name in s.dev:
        s.dev[name].copy_(t.dev[name])
    s.mask.copy_(t.mask)
    q.copy_(torch.randn_like(q))
    w1.fill_(255)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    check(og, lg, t.ref(q, k64, v64, 0.1), 128, 1250)
    assert torch.equal(og, oh) and torch.equal(lg, lh)


@KINDS
def test_cache_beyond_two_giga_elements(quant):
    """Cache rows whose offsets pass 32 bits."""
    Hkv, d = 8, 128
    rows = ((1 << 31) // (Hkv * d) + 1024) // 64 * 64
    s = Step(14, [2, 9], [100, 700], 64)
    q, kt, vt, scales, k64, v64 = make(14, s.N, s.rows, 16, Hkv, d, quant)
    u8 = (lambda t: t.view(torch.uint8)) if quant else (lambda t: t)
    k = torch.empty((rows, Hkv, d), dtype=u8(kt).dtype, device="cuda")
    v = torch.empty_like(k)
    k[-s.rows:], v[-s.rows:] = u8(kt), u8(vt)
    if quant:
        wide = {n: torch.empty((Hkv, rows), device="cuda") for n in scales}
        for n in scales:
            wide[n][:, -s.rows:] = scales[n]
        scales = wide
    ref = s.ref(q, k64, v64, 0.1)
    s.dev["page_table"] += (rows - s.rows) // 64
    o, lse, _ = s.call(q, k.view(kt.dtype), v.view(vt.dtype), 0.1, **scales)
    check(o, lse, ref, d, 710)


@KINDS
@pytest.mark.parametrize("nodes", [1, 30])
def test_what_does_not_fit_is_reported(nodes, quant):
    """Lengths, rows and pages outside their arrays: nothing outside the outputs is written, and
    the other requests' rows are right."""
    s = Step(15, [nodes] * 3, [200, 150, 90], 16)
    q, k, v, scales, k64, v64 = make(15, s.N, s.rows, 8, 2, 128, quant)
    ref = s.ref(q, k64, v64, 0.1)
    table = s.dev["page_table"]
    pages = s.rows // 16
    bad_pages = [table.clone() for _ in range(4)]
    for t, x in zip(bad_pages, (-1, pages, 2 ** 31 - 1, -2 ** 31)):
        t[1, 3] = x
    cases = [dict(page_table=t) for t in bad_pages] + [
        dict(kv_lens=i32([200, x, 90])) for x in (-1, 16 * table.shape[1], 2 ** 31 - 1, -2 ** 31)] + [
        dict(q_start=i32([0, nodes, 10 ** 6, 3 * nodes])), dict(q_start=i32([0, nodes, -5, 3 * nodes]))]
    for kw in cases:
        og, lg = Guarded((s.N, 8, 128), torch.bfloat16, 9.0), Guarded((s.N, 8), torch.float32, 9.0)
        status = cpa.new_status()
        dev, s.dev = s.dev, {**s.dev, **kw}
        s.call(q, k, v, 0.1, out=og.t, lse=lg.t, status=status, **scales)
        s.dev = dev
        for x in (og, lg):
            x.check(str(kw))
        assert int(status.item()) == L.ERR_RANGE, kw
        fine = list(range(nodes)) + ([] if "q_start" in kw else list(range(2 * nodes, s.N)))
        check(og.t[fine], lg.t[fine], {n: x[fine] for n, x in ref.items()}, 128, 260)
    # more rows than the mask has bits for
    if nodes > 1:
        many = Step(16, [40, 2], [20, 30], 16)
        q, k, v, scales, _, _ = make(16, 42, many.rows, 8, 2, 128, quant)
        status = cpa.new_status()
        many.call(q, k, v, 0.1, mask=many.mask[:, :1].contiguous(), status=status, **scales)
        assert int(status.item()) == L.ERR_RANGE


@KINDS
@pytest.mark.parametrize("nodes", [1, 4, 8, 30, 64])
def test_a_wait_that_runs_out_is_reported(nodes, quant):
    """With the queries never published, the waits on them run out in every kernel: it is
    reported, the copies are drained, and the same call is right afterwards."""
    lib = L.load()
    s = Step(17, [nodes, nodes], [900, 700], 16)
    q, k, v, scales, k64, v64 = make(17, s.N, s.rows, 8, 2, 128, quant)
    status = cpa.new_status()
    call = lambda: s.call(q, k, v, 0.1, num_ctas=7, status=status, **scales)  # noqa: E731
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
    check(o, lse, s.ref(q, k64, v64, 0.1), 128, 970)


@KINDS
def test_steps_of_a_drafting_server(quant):
    """Append, layout, rotation and attention together, as a server with drafted trees uses
    them: each step's trees go behind the cached keys, their rows attend, and of each tree
    the path to one node is kept."""
    Hq, Hkv, d, page, B, T = 8, 2, 64, 16, 3, 6
    rng = random.Random(18)
    g = torch.Generator(device="cuda").manual_seed(18)
    r = lambda *x: torch.randn(x, generator=g, device="cuda").bfloat16()  # noqa: E731
    inv_freq = 10000.0 ** (-np.arange(32) / 32)
    rope = cpa.make_rope(inv_freq)
    rows, width = 20 * page, 6
    pages = list(range(20))
    rng.shuffle(pages)
    table = [pages[b * width: (b + 1) * width] for b in range(B)]
    page_table, q_start = i32(table), i32([T * b for b in range(B + 1)])
    cache = cpa.alloc_kv_cache(rows, Hkv, d, d) if quant else \
        tuple(torch.zeros((rows, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc, vc = (cache.k, cache.v) if quant else cache
    kw = dict(k_scale=cache.k_scale, v_scale=cache.v_scale) if quant else {}
    kv, status = [0, 0, 0], cpa.new_status()
    ws = cpa.alloc_tree_workspace(Hq, Hkv, d, T)
    for step in range(4):
        parents = [rng.randint(max(-1, i - 3), i - 1) for _ in range(B) for i in range(T)]
        slots, positions, mask = cpa.cp_tree_layout(q_start, i32(kv), page_table, page, B * T, parents=i32(parents),
                                                    max_nodes=T, status=status)
        q, k, v = r(B * T, Hq, d), r(B * T, Hkv, d), r(B * T, Hkv, d)
        pos = positions.cpu().numpy()[None]
        before = q.clone()
        cpa.cp_kv_append(cache, k, v, slots, rope=rope, positions=positions, q=q, out_q=q, status=status)
        o, lse, _ = cpa.cp_attn_tree(q, kc, vc, page_table, page, q_start, i32(kv), d ** -0.5, mask=mask,
                                     max_nodes=T, workspace=ws, status=status, **kw)
        cpa.check_status(status)
        # the rotated rows are within their rounding of the oracle's; from there on as cached
        want = op.rotate(f64(before), pos, inv_freq)
        assert (np.abs(f64(q) - want) <= 2.0 ** -7 * np.abs(want).max()).all()
        k64, v64 = (f64(x) for x in (cpa.cp_kv_dequantize(cache, out_fp32=True) if quant else cache))
        at = slots.tolist()
        assert (np.abs(k64[at] - op.rotate(f64(k), pos, inv_freq)) <= (2.0 ** -4 if quant else 2.0 ** -7) *
                np.abs(f64(k)).max(-1, keepdims=True) * 1.5).all()
        _, want_pos, seen = op.tree_layout(list(range(0, B * T + 1, T)), kv, table, page, parents, B * T)
        assert want_pos == positions.tolist()
        ref = op.tree_attention(f64(q), k64, v64, list(range(0, B * T + 1, T)), kv, table, page, seen, d ** -0.5)
        check(o, lse, ref, d, 60, f"step {step}")
        # keep a path of each tree: its keys move up behind the cached ones, positions and all
        src, dst = [], []
        for b in range(B):
            kept = np.nonzero(seen[b][rng.randrange(T)])[0]
            for i, node in enumerate(kept):
                src.append(at[b * T + int(node)])
                dst.append(table[b][(kv[b] + i) // page] * page + (kv[b] + i) % page)
                assert want_pos[b * T + int(node)] == kv[b] + i
            kv[b] += len(kept)
        for t in (kc, vc):
            t = t.view(torch.uint8) if quant else t
            t[dst] = t[src]
        for x in kw.values():
            x[:, dst] = x[:, src]


def test_refusals_of_the_binding():
    s = Step(19, [2, 3], [10, 20], 16)
    q, k, v, scales, _, _ = make(19, s.N, s.rows, 8, 2, 128, True)
    kb = torch.zeros((s.rows, 2, 128), dtype=torch.bfloat16, device="cuda")
    for kw, err in ((dict(k_scale=scales["k_scale"]), ValueError), ({}, TypeError)):
        with pytest.raises(err):
            s.call(q, k, v, 0.1, **kw)
    for a, err in (((q, kb, kb[:16]), ValueError), ((q, kb[:, :, :64], kb), ValueError), ((q.float(), kb, kb), TypeError),
                   ((q[:, :7], kb, kb), L.CpAttnError), ((q[:3], kb, kb), ValueError)):
        with pytest.raises(err):
            s.call(*a, 0.1)
    for kw, err in ((dict(mask=s.mask[:3]), ValueError), (dict(mask=s.mask.long()), TypeError),
                    (dict(max_nodes=0), L.CpAttnError), (dict(num_ctas=0), L.CpAttnError),
                    (dict(out=torch.empty(5, 8, 64, device="cuda")), ValueError),
                    (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), L.CpAttnError)):
        with pytest.raises(err):
            s.call(q, kb, kb, 0.1, **kw)
    for name, x in (("kv_lens", i32([1])), ("q_start", i32([0, 5])), ("page_table", i32([[1]])),
                    ("page_table", s.dev["page_table"].long())):
        dev, s.dev = s.dev, {**s.dev, name: x}
        with pytest.raises((ValueError, TypeError)):
            s.call(q, kb, kb, 0.1)
        s.dev = dev
    s.page = 24
    with pytest.raises(L.CpAttnError):
        s.call(q, kb, kb, 0.1)


@KINDS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [1, 3, 12, 40])
def test_long_batches_again_and_again(nodes, d, quant):
    """Many pieces and tiles a block, all of its warps and rings going round many times, at
    rates that memory sets: no wait runs out, and every call gives the same bits."""
    B, Hq, Hkv = 40, 32, 32 if nodes == 1 else 8
    rng = random.Random(20)
    kv = [rng.randint(0, 4000) for _ in range(B)]
    s = Step(20, [nodes] * B, kv, 16)
    q, k, v, scales, _, _ = make(20, s.N, 64, Hq, Hkv, d, quant)
    big = lambda t: t.repeat(-(-s.rows // 64), 1, 1)[: s.rows].contiguous()  # noqa: E731
    k, v = (big(t.view(torch.uint8)).view(t.dtype) if quant else big(t) for t in (k, v))
    scales = {n: x.repeat(1, -(-s.rows // 64))[:, : s.rows].contiguous() for n, x in scales.items()}
    status = cpa.new_status()
    ws = cpa.alloc_tree_workspace(Hq, Hkv, d, nodes)
    first = None
    for _ in range(12):
        o, lse, _ = s.call(q, k, v, 0.1, workspace=ws, status=status, **scales)
        first = (o, lse) if first is None else first
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    cpa.check_status(status)
