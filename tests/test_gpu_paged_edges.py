"""Calls of a paged decode step that the documentation allows and that take a way of their
own: queries that no box holds, scales that no 16-byte copy takes, pages that requests share,
buffers that a call on another stream makes.  Tolerances are those of test_gpu_tree."""

import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L
from context_causal_attention_cp_gb300 import api
from oracle import paged as op

import test_gpu_rope as rotation
from test_gpu_guards import Guarded
from test_gpu_shared import check, f64, make
from test_gpu_tree import KINDS, Step, i32

pytestmark = pytest.mark.gpu


@KINDS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(6, 2), (20, 4), (14, 2)], ids=["g3", "g5", "g7"])
@pytest.mark.parametrize("nodes", [[20, 11], [64, 50]], ids=["single", "dual"])
def test_groups_that_do_not_divide_a_tile(nodes, heads, d, quant):
    Hq, Hkv = heads
    s = Step(Hq, nodes, [200, 77], 32)
    q, k, v, scales, k64, v64 = make(Hq, s.N, s.rows, Hq, Hkv, d, quant)
    o, lse, _ = s.call(q, k, v, d ** -0.5, **scales)
    check(o, lse, s.ref(q, k64, v64, d ** -0.5), d, 277)


@KINDS
@pytest.mark.parametrize("nodes", [[2, 1], [20, 11], [64, 50]], ids=["small", "single", "dual"])
def test_queries_shared_by_heads_or_rows(nodes, quant):
    """q expanded: one vector for all heads of a row, or for all rows."""
    Hq, Hkv, d = 8, 2, 128
    s = Step(5, nodes, [150, 40], 16)
    q, k, v, scales, k64, v64 = make(5, s.N, s.rows, Hq, Hkv, d, quant)
    for x in (q[:, :1].expand(-1, Hq, -1), q[:1].expand(s.N, -1, -1), q[:1, :1].expand(s.N, Hq, -1)):
        o, lse, _ = s.call(x, k, v, 0.1, **scales)
        check(o, lse, s.ref(x, k64, v64, 0.1), d, 214)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [[2, 1, 1], [20, 11, 3], [64, 50, 7]], ids=["small", "single", "dual"])
def test_scales_at_any_word(nodes, d):
    """Scale rows that start at a 4-byte boundary, and rows of an odd stride."""
    Hq, Hkv = 8, 2
    s = Step(6, nodes, [300, 17, 129], 16)
    q, k, v, scales, k64, v64 = make(6, s.N, s.rows, Hq, Hkv, d, True, 2.0)
    want = s.call(q, k, v, 0.1, **scales)
    ref = s.ref(q, k64, v64, 0.1)
    for pad in (1, 2, 4):
        moved = {}
        for name, x in scales.items():
            wide = torch.full((Hkv, s.rows + pad), float("nan"), device="cuda")
            wide[:, pad:] = x
            moved[name] = wide[:, pad:]
        o, lse, _ = s.call(q, k, v, 0.1, **moved)
        check(o, lse, ref, d, 364)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@KINDS
def test_requests_that_share_pages(quant):
    """A prompt's pages in the tables of all requests, each with pages of its own behind."""
    Hq, Hkv, d, page, prompt = 8, 2, 128, 16, 160
    nodes, kv = [1, 5, 2], [prompt + 3, prompt, prompt + 20]
    s = Step(8, nodes, kv, page)
    for b in (1, 2):
        s.table[b][: prompt // page] = s.table[0][: prompt // page]
    s.dev["page_table"] = i32(s.table)
    q, k, v, scales, k64, v64 = make(8, s.N, s.rows, Hq, Hkv, d, quant)
    o, lse, _ = s.call(q, k, v, 0.1, **scales)
    check(o, lse, s.ref(q, k64, v64, 0.1), d, 190)


@KINDS
@pytest.mark.parametrize("nodes", [1, 20, 64])
def test_two_calls_at_once(nodes, quant):
    """Two batches on two streams with a workspace each give what they give alone."""
    Hq, Hkv, d = 32, 8, 128
    both = []
    for seed in (1, 2):
        s = Step(seed, [nodes] * 12, [700 * seed + 31 * b for b in range(12)], 16)
        q, k, v, scales, _, _ = make(seed, s.N, s.rows, Hq, Hkv, d, quant)
        both.append((s, (q, k, v, 0.1), dict(scales, workspace=cpa.alloc_tree_workspace(Hq, Hkv, d, nodes))))
    want = [tuple(t.clone() for t in s.call(*a, **kw)[:2]) for s, a, kw in both]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(5):
        got = []
        for (s, a, kw), stream in zip(both, streams):
            got.append(s.call(*a, stream=stream, **kw)[:2])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_a_table_that_is_expanded_is_refused():
    s = Step(9, [1, 1], [20, 20], 16)
    q, k, v, _, _, _ = make(9, s.N, s.rows, 8, 2, 128, False)
    s.dev["page_table"] = s.dev["page_table"][:1].expand(2, -1)
    with pytest.raises(L.CpAttnError):
        s.call(q, k, v, 0.1)


def test_nothing_to_do():
    """No rows, no requests, or rows that are all padding: outputs stay as they are."""
    none = Step(10, [], [], 16, width=4)
    q, k, v, _, _, _ = make(10, 3, 32, 8, 2, 128, False)
    empty = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    at, lens = i32([0]), torch.empty(0, dtype=torch.int32, device="cuda")
    out, lse = torch.full((3, 8, 128), 3.0, device="cuda"), torch.full((3, 8), 4.0, device="cuda")
    cpa.cp_attn_tree(q, k, v, empty, 16, at, lens, 0.1, out=out, lse=lse)
    cpa.cp_attn_tree(q[:0], k, v, empty, 16, at, lens, 0.1)
    two = dict(page_table=i32([[0, 1], [1, 0]]), q_start=i32([0, 0, 0]), kv_lens=i32([20, 0]))
    cpa.cp_attn_tree(q, k, v, two["page_table"], 16, two["q_start"], two["kv_lens"], 0.1, out=out, lse=lse)
    slots, positions, mask = cpa.cp_tree_layout(at, lens, empty, 16, 3, parents=i32([-1] * 3), max_nodes=1)
    assert slots.tolist() == [-1] * 3 and positions.tolist() == [0] * 3 and not mask.any()
    cpa.cp_kv_append((k, v), k[:3], v[:3], slots)
    cpa.cp_kv_append((k, v), k[:0], v[:0])
    rope = cpa.make_rope([1.0] * 8)
    assert cpa.cp_rope(rope, q[:0], positions=at[:0])[0].shape == (0, 8, 128)
    assert (out == 3.0).all() and (lse == 4.0).all() and none.N == 0


CALLS = ("rope", "append", "layout", "attn")


@pytest.mark.parametrize("name", CALLS)
def test_buffers_belong_to_the_calls_stream(name, monkeypatch):
    s = Step(12, [3, 2], [20, 33], 16)
    q, k, v, _, _, _ = make(12, s.N, s.rows, 8, 2, 128, False)
    rope = cpa.make_rope([1.0 / (1 + c) for c in range(32)])
    at, parents = i32(s.positions), i32(s.parents)
    call = {
        "rope": lambda **kw: cpa.cp_rope(rope, q, q[:, :2], at, **kw),
        "append": lambda **kw: (cpa.cp_kv_append((k.clone(), v.clone()), q[:, :2], q[:, 2:4], i32(s.slots), rope=rope,
                                                 positions=at, q=q, **kw),),
        "layout": lambda **kw: cpa.cp_tree_layout(s.dev["q_start"], s.dev["kv_lens"], s.dev["page_table"], 16, s.N,
                                                  parents=parents, max_nodes=3, **kw),
        "attn": lambda **kw: s.call(q, k, v, 0.1, **kw)[:2],
    }[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made, empty = [], torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        if t.is_cuda:
            made.append(torch.cuda.current_stream().cuda_stream)
        return t

    if name == "append":  # (its own copies are made here, before the other stream's work)
        kc, vc, slots = k.clone(), v.clone(), i32(s.slots)
        torch.cuda.synchronize()
        call = lambda **kw: (cpa.cp_kv_append((kc, vc), q[:, :2], q[:, 2:4], slots, rope=rope,  # noqa: E731
                                              positions=at, q=q, **kw),)
    monkeypatch.setattr(api.torch, "empty", spy)
    got = call(stream=side)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert made and set(made) == {side.cuda_stream}
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_rotation_before_or_with_the_append():
    """Rotating first and appending then gives what one call gives, but for K's rounding in
    between, and Q's is the same call."""
    n, Hq, Hkv, d = 37, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((n, h, d), generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    rope = cpa.make_rope([10000.0 ** (-c / 64) for c in range(64)])
    at = torch.randint(0, 5000, (n,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(64, generator=g, device="cuda")[:n].int()
    caches = [tuple(torch.zeros((64, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)) for _ in range(2)]
    qr, kr = cpa.cp_rope(rope, q, k, at)
    cpa.cp_kv_append(caches[0], kr, v, slots)
    qa = cpa.cp_kv_append(caches[1], k, v, slots, rope=rope, positions=at, q=q)
    assert torch.equal(qa, qr)
    for a, b in zip(*caches):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n, Hq, d, pairs, first", [
    (600, 2, 1024, 512, 0), (300, 1, 768, 384, 0), (700, 1, 768, 384, 0), (500, 3, 576, 32, 512), (457, 1, 16, 8, 0),
    (456, 40, 16, 8, 0), (1000, 48, 64, 32, 0), (2000, 3, 272, 8, 256), (9000, 1, 512, 256, 0)])
def test_rows_on_both_sizes_of_blocks(n, Hq, d, pairs, first, dtype):
    """Wide and narrow vectors, one and many a row, at numbers of rows that take blocks of
    either size and rows that end inside a block."""
    rope, pos, rot, ref = rotation.make(n, n, pairs, 2, first, n % 2 == 1)
    x = rotation.draw(n, (n, Hq, d), dtype)
    out, status = Guarded((n, Hq, d), dtype), cpa.new_status()
    cpa.cp_rope(rope, x, positions=pos, out_q=out.t, status=status)
    cpa.check_status(status)
    out.check("q")
    rotation.check(out.t, x, rot, op.rotate(f64(x), **ref))
    # the same rows into a cache, backwards
    cache = (torch.zeros((n + 3, Hq, d), dtype=torch.bfloat16, device="cuda"), None)
    slots = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    cpa.cp_kv_append(cache, x, None, slots, rope=rope, positions=pos, status=status)
    cpa.check_status(status)
    assert torch.equal(cache[0][:n].flip(0), out.t.bfloat16()) and not cache[0][n:].any()


@KINDS
@pytest.mark.parametrize("d", [64, 128])
def test_any_number_of_nodes_to_tune_for_and_of_blocks(d, quant):
    """Units of every size on rows that they were not chosen for, on one block and on more than
    the device has."""
    Hq, Hkv = 8, 2
    s = Step(14, [1, 30, 0, 7, 1], [700, 60, 5, 0, 128], 32)
    q, k, v, scales, k64, v64 = make(14, s.N, s.rows, Hq, Hkv, d, quant)
    ref = s.ref(q, k64, v64, 0.1)
    for most in (1, 2, 4, 5, 32, 33, 100000):
        for ctas in (1, 2, 7, 152, 4096):
            status = cpa.new_status()
            o, lse, _ = s.call(q, k, v, 0.1, max_nodes=most, num_ctas=ctas, status=status, **scales)
            cpa.check_status(status, f"{most} nodes, {ctas} blocks")
            check(o, lse, ref, d, 701, f"{most} nodes, {ctas} blocks")


@KINDS
@pytest.mark.parametrize("nodes", [[2, 1], [20, 11], [64, 50]], ids=["small", "single", "dual"])
def test_a_page_of_65536_rows_and_an_output_at_16_bytes(nodes, quant):
    Hq, Hkv, d = 4, 1, 64
    s = Step(15, nodes, [300, 777], 65536, spare=0)
    q, k, v, scales, k64, v64 = make(15, s.N, s.rows, Hq, Hkv, d, quant)
    room = torch.full((s.N * Hq * d + 16,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = room[8:-8].view(s.N, Hq, d)
    assert out.data_ptr() % 32 == 16
    o, lse, _ = s.call(q, k, v, 0.1, out=out, **scales)
    check(o, lse, s.ref(q, k64, v64, 0.1), d, 827)
    assert (room[:8] == 5.0).all() and (room[-8:] == 5.0).all()


def test_k_that_is_v_too():
    s = Step(16, [3, 9], [200, 31], 16)
    q, k, _, _, k64, _ = make(16, s.N, s.rows, 8, 2, 128, False)
    o, lse, _ = s.call(q, k, k, 0.1)
    check(o, lse, s.ref(q, k64, k64, 0.1), 128, 203)


def test_positions_that_axes_share():
    """Positions expanded over the axes, cut out of a longer row, or one row's of a table."""
    n, d = 70, 96
    rope, _, rot, ref = rotation.make(3, n, 24, 3)
    x, cache = rotation.draw(4, (n, 2, d), torch.bfloat16), torch.zeros((n, 2, d), dtype=torch.bfloat16, device="cuda")
    long = torch.arange(5000, 5000 + 3 * n, dtype=torch.int32, device="cuda")
    wide = torch.stack([long, long + 7, long * 3])
    for pos in (long[5:5 + n].expand(3, n), wide[:, 9:9 + n], long.view(n, 3).t().contiguous(), wide[:, 30:31].expand(3, n)[:, :1]):
        m = pos.shape[1]
        want = op.rotate(f64(x[:m]), **{**ref, "positions": pos.cpu().numpy()})
        got, _ = cpa.cp_rope(rope, x[:m], positions=pos)
        rotation.check(got, x[:m], rot, want)
        cpa.cp_kv_append((cache, None), x[:m], None, rope=rope, positions=pos)
        assert torch.equal(cache[:m], got)
    with pytest.raises(ValueError):
        cpa.cp_rope(rope, x, positions=long.view(n, 3).t())


@pytest.mark.parametrize("nodes", [20, 64], ids=["single", "dual"])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_many_sizes_in_short_pieces(d, nodes):
    """Requests of a tile or two whose queries differ by 2^50, many to a block: each piece's
    scores go by the exponents of its own queries."""
    Hq, Hkv, B = 8, 2, 48
    kv = [(37 * b) % 200 for b in range(B)]
    s = Step(21, [nodes] * B, kv, 16)
    q, k, v, scales, k64, v64 = make(21, s.N, s.rows, Hq, Hkv, d, True)
    up = torch.tensor([25 - 50 * (b % 2) for b in range(B)], device="cuda").repeat_interleave(nodes)
    q = (q.float() * torch.exp2(up.float())[:, None, None]).bfloat16()
    ref = s.ref(q, k64, v64, 2.0 ** -25)
    for ctas in (1, 2, 8, 152):
        o, lse, _ = s.call(q, k, v, 2.0 ** -25, num_ctas=ctas, **scales)
        check(o, lse, ref, d, 264, f"{ctas} blocks")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotated_into_the_slot_beside(dtype):
    """Q and K of a buffer [rows, heads, 3, d] into its other slots, which no other element meets."""
    n, H, d = 300, 5, 64
    rope, pos, rot, ref = rotation.make(22, n, 32)
    both = rotation.draw(23, (n, H, 3, d), dtype)
    before = both.clone()
    cpa.cp_rope(rope, both[:, :, 0], positions=pos, out_q=both[:, :, 2])
    rotation.check(both[:, :, 2], before[:, :, 0], rot, op.rotate(f64(before[:, :, 0]), **ref))
    assert torch.equal(both[:, :, :2], before[:, :, :2])
    with pytest.raises(L.CpAttnError):
        cpa.cp_rope(rope, both[1:, :, 0], positions=pos[:, 1:], out_q=both[:-1, :, 0])
