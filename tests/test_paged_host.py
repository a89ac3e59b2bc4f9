"""Host side of rotary positions, of the cache's append and of a decode step over a paged
cache: bad arguments are refused before anything is launched, the bindings' argument
structures are C's, and the oracle's own parts agree with plain formulas.  No GPU."""

import copy
import ctypes
import math
import os
import pickle
import shutil
import subprocess

import numpy as np
import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L
from oracle import paged as op

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, KIND, ALIGN, LARGE = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED, L.ERR_ALIGNMENT, L.ERR_TOO_LARGE


def refused(call, cases):
    for want, kws in cases.items():
        for kw in kws:
            assert call(**kw) == want, (want, kw)


def rope_of(**kw):
    return L.RopeInfo(**{**dict(table=0x900000, pairs=32, first=0, interleaved=0, axes=1), **kw})


ROPE = dict(q=0x10000, k=0x200000, qo=0x400000, ko=0x600000, at=0x800000, status=0, qr=512, qh=128, kr=256, kh=128,
            qor=512, qoh=128, kor=256, koh=128, axis=0, n=8, Hq=4, Hk=2, d=128, f32=0, inverse=0)


def call_rope(rope=rope_of(), **kw):
    assert set(kw) <= set(ROPE)
    return L.load().cp_rope(rope, L.ROPE_ARGS.pack(*{**ROPE, **kw}.values()), None)


def test_rope_refusals():
    refused(call_rope, {
        BAD: (dict(rope=None), dict(rope=rope_of(pairs=0)), dict(rope=rope_of(pairs=-8)), dict(rope=rope_of(first=-8)),
              dict(rope=rope_of(axes=0)), dict(rope=rope_of(axes=9)), dict(rope=rope_of(first=72)),
              dict(rope=rope_of(first=2 ** 31 - 8)), dict(rope=rope_of(pairs=72)), dict(rope=rope_of(table=None)),
              dict(rope=rope_of(axes=2), axis=-1), dict(at=0), dict(q=0), dict(qo=0), dict(k=0), dict(ko=0), dict(n=-1),
              dict(Hq=0), dict(Hk=-1), dict(Hq=1 << 21), dict(Hk=1 << 21), dict(qr=-8), dict(kh=-8), dict(qor=0), dict(koh=0),
              dict(qoh=120), dict(kor=248),
              # outputs that meet their inputs
              dict(qo=0x10000 + 256), dict(qo=0x10000 - 4096), dict(qo=0x10000, qor=1024), dict(ko=0x200000 + 128)),
        KIND: (dict(rope=rope_of(pairs=12)), dict(rope=rope_of(first=4)), dict(d=8), dict(d=1040), dict(d=120)),
        ALIGN: (dict(q=0x10008), dict(qo=0x400008), dict(ko=0x600004), dict(qr=516), dict(koh=132), dict(f32=1, qh=130),
                dict(at=0x800002), dict(status=0x700001), dict(rope=rope_of(table=0x900008))),
        LARGE: (dict(qr=1 << 37, qo=1 << 45), dict(kh=1 << 36, f32=1, ko=1 << 45), dict(qor=1 << 37)),
        L.OK: (dict(n=0, q=0, k=0, qo=0, ko=0, at=0), dict(n=0, Hk=0, k=0, ko=0),
               dict(n=0, qor=0, qoh=0, kor=0, koh=0)),
    })


def test_rope_table():
    lib = L.load()
    f = (ctypes.c_double * 4)(1.0, 0.25, 2 * math.pi, 0.0)
    ax = (ctypes.c_int32 * 4)(0, 1, 7, 0)
    t = (ctypes.c_int32 * 16)()
    assert lib.cp_rope_table(f, ax, 4, t) == L.OK
    for c in range(4):
        F = (t[4 * c] & 0xffffffff) | (t[4 * c + 1] & 0xffffffff) << 32
        turns = f[c] / (2 * math.pi)
        off = (F / 2.0 ** 64 - turns + 0.5) % 1 - 0.5
        assert abs(off) < 2.0 ** -52 and t[4 * c + 2] == ax[c] and t[4 * c + 3] == 0
    for bad in (float("nan"), float("inf"), 2.0 ** 21):
        assert lib.cp_rope_table((ctypes.c_double * 1)(bad), None, 1, t) == BAD
    for a in (-1, 8):
        assert lib.cp_rope_table(f, (ctypes.c_int32 * 1)(a), 1, t) == BAD
    for n in (0, -1, 513):
        assert lib.cp_rope_table(f, None, n, t) == BAD
    assert lib.cp_rope_table(None, None, 1, t) == BAD and lib.cp_rope_table(f, None, 1, None) == BAD


@pytest.mark.parametrize("f", [1.0, 0.73, 1e-4, 1000.5, -2.25, 2.0 ** 20])
def test_rope_table_keeps_far_positions(f):
    """A position times the table's fraction is the oracle's angle, to 2^-64 turns a position
    and the oracle's double (2 pi 2^-53)."""
    t = (ctypes.c_int32 * 4)()
    assert L.load().cp_rope_table((ctypes.c_double * 1)(f), None, 1, t) == L.OK
    F = (t[0] & 0xffffffff) | (t[1] & 0xffffffff) << 32
    for at in (1, 1000, 123456789, 2 ** 31 - 1, -5, -2 ** 31):
        got = 2 * math.pi * ((at * F) % 2 ** 64) / 2.0 ** 64
        want = op.angles([[at]], [f], [0])[0, 0]
        off = (got - want + math.pi) % (2 * math.pi) - math.pi
        # an angle that the oracle leaves unreduced, x = at f, costs here: the sums got - x + pi a
        # rounding each, at most 2^-53 |x| (1 + pi / |x|), and x / 2 pi turns the error of pi's
        # double, at most 2^-53 |x|; together at most 2^-53 (3 |x| + 4 pi)
        x = abs(at * f) if abs(at) < 1 << 20 else 0
        bound = 2 * math.pi * (abs(at) * 2.0 ** -64 + 4 * 2.0 ** -53) + 2.0 ** -53 * (3 * x + 4 * math.pi)
        assert abs(off) <= bound, (f, at, off, bound)


APPEND = dict(k=0x10000, v=0x100000, q=0x200000, qo=0x300000, at=0x800000, slots=0x810000, status=0, kr=256, kh=128, vr=256,
              vh=128, qr=512, qh=128, qor=512, qoh=128, axis=0, n=8, Hkv=2, d=128, dv=128, Hq=4, rows=64, f32=0)


def codes(**kw):
    return L.KvCodes(**{**dict(codes=0x500000, scales=0x600000, row_stride=256, head_stride=128, scale_stride=64), **kw})


def rows(**kw):
    return codes(**{**dict(scales=None, row_stride=512, head_stride=256, scale_stride=0), **kw})


def call_append(rope=rope_of(), kc=codes(), vc=codes(codes=0x700000, scales=0x780000), **kw):
    assert set(kw) <= set(APPEND)
    kc, vc = (None if c is None else ctypes.byref(c) for c in (kc, vc))
    return L.load().cp_kv_append(rope, kc, vc, L.KV_APPEND_ARGS.pack(*{**APPEND, **kw}.values()), None)


def test_append_refusals():
    refused(call_append, {
        BAD: (dict(kc=None), dict(vc=None), dict(v=0), dict(k=0), dict(n=-1), dict(rows=-1), dict(Hkv=0), dict(Hkv=1 << 21),
              dict(Hq=-1), dict(Hq=1 << 21), dict(q=0), dict(qo=0), dict(at=0), dict(kr=-8), dict(vh=-8), dict(qh=-8),
              dict(rows=65), dict(kc=codes(codes=None)), dict(kc=codes(scales=None)), dict(vc=rows()),
              dict(kc=codes(head_stride=112)), dict(kc=codes(row_stride=240)), dict(kc=codes(scale_stride=63)),
              dict(kc=rows(row_stride=256), vc=rows()), dict(kc=rows(), vc=rows(head_stride=240)),
              dict(qo=0x200000 + 256), dict(rope=rope_of(pairs=72)), dict(rope=rope_of(axes=3), axis=-8),
              dict(rope=rope_of(table=None))),
        KIND: (dict(d=120), dict(d=8, rope=None), dict(dv=1040), dict(dv=0), dict(rope=rope_of(pairs=4))),
        ALIGN: (dict(k=0x10008), dict(v=0x100002), dict(q=0x200008), dict(qo=0x300008), dict(slots=0x810002),
                dict(status=0x900001), dict(at=0x800002), dict(kr=260), dict(vh=132), dict(f32=1, kh=130),
                dict(kc=codes(codes=0x500008)), dict(vc=codes(scales=0x600002)), dict(kc=codes(row_stride=264)),
                dict(kc=rows(head_stride=264), vc=rows())),
        LARGE: (dict(kr=1 << 37), dict(kc=codes(row_stride=1 << 37)), dict(qor=1 << 37)),
        L.OK: (dict(n=0), dict(n=0, rope=None, at=0), dict(n=0, k=0, v=0, q=0, qo=0, slots=0),
               dict(n=0, kc=rows(), vc=rows()), dict(n=0, v=0, vc=None, dv=0)),
    })


LAYOUT = dict(q_start=0x10000, kv_lens=0x20000, table=0x30000, parents=0x40000, slots=0x50000, positions=0x60000,
              mask=0x70000, status=0, stride=8, reqs=2, pages=8, page=16, n=5, words=1)


def test_layout_refusals():
    def call(**kw):
        assert set(kw) <= set(LAYOUT)
        return L.load().cp_tree_layout(L.TREE_LAYOUT_ARGS.pack(*{**LAYOUT, **kw}.values()), None)

    assert L.load().cp_tree_layout(None, None) == BAD
    refused(call, {
        BAD: (dict(q_start=0), dict(kv_lens=0), dict(table=0), dict(slots=0), dict(positions=0), dict(mask=0),
              dict(parents=0), dict(words=0), dict(words=-1), dict(parents=0, mask=0, words=-1), dict(reqs=-1),
              dict(reqs=1 << 24), dict(n=-1), dict(pages=-1), dict(stride=7)),
        KIND: (dict(page=0), dict(page=8), dict(page=24), dict(page=-16), dict(page=1 << 17)),
        ALIGN: (dict(q_start=0x10002), dict(kv_lens=0x20001), dict(table=0x30002), dict(parents=0x40002),
                dict(slots=0x50001), dict(positions=0x60002), dict(mask=0x70001), dict(status=0x80002)),
        L.OK: (dict(n=0), dict(n=0, slots=0, positions=0, q_start=0)),
    })


ATTN = dict(q=0x10000, k=0x100000, v=0x200000, ks=0, vs=0, table=0x300000, q_start=0x310000, kv_lens=0x320000, mask=0x330000,
            o=0x400000, lse=0x500000, ws=0x600000, status=0, qr=1024, qh=128, kr=256, kh=128, vr=256, vh=128, ss=0,
            stride=8, nb=0, n=5, rows=256, pages=8, page=16, reqs=2, words=1, Hq=8, Hkv=2, d=128, dv=128, nodes=4,
            ctas=152, f32=0, scale=0.1)


def test_attention_refusals():
    need = cpa.cp_tree_workspace_size(8, 2, 128, 4, 152)

    def call(**kw):
        assert set(kw) <= set(ATTN)
        return L.load().cp_attn_tree(L.ATTN_TREE_ARGS.pack(*{**ATTN, "nb": need, **kw}.values()), None)

    assert L.load().cp_attn_tree(None, None) == BAD
    quant = dict(ks=0x700000, vs=0x780000, ss=256)
    refused(call, {
        BAD: (dict(q=0), dict(k=0), dict(v=0), dict(table=0), dict(q_start=0), dict(kv_lens=0), dict(o=0), dict(lse=0),
              dict(ws=0), dict(nb=need - 1), dict(mask=0), dict(words=0), dict(words=-1), dict(n=-1), dict(rows=-1),
              dict(rows=15), dict(reqs=-1), dict(reqs=1 << 24), dict(pages=0), dict(pages=-1), dict(stride=7),
              dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(Hq=0), dict(Hkv=0), dict(Hq=7),
              dict(Hq=1 << 21), dict(nodes=0), dict(ctas=0), dict(ctas=4097), dict(qr=-8), dict(qh=-8), dict(kr=248),
              dict(kh=120), dict(vr=248), dict(vh=64), {**quant, "ks": 0}, {**quant, "vs": 0}, {**quant, "ss": 255}),
        KIND: (dict(d=64), dict(dv=64), dict(d=96, dv=96), dict(d=256, dv=256), dict(page=8), dict(page=24), dict(page=0),
               dict(page=-16), dict(page=1 << 17)),
        ALIGN: (dict(q=0x10008), dict(k=0x100008), dict(v=0x200008), dict(o=0x400008), dict(ws=0x600010),
                dict(lse=0x500002), dict(table=0x300002), dict(q_start=0x310001), dict(kv_lens=0x320002),
                dict(mask=0x330002), dict(status=0x340002), dict(qr=1028), dict(qh=132), dict(kr=260), dict(vh=132),
                {**quant, "kr": 264}, {**quant, "ks": 0x700002}, {**quant, "vs": 0x700001}),
        LARGE: (dict(n=2 ** 31 - 1, qr=128, Hq=8),),
        L.OK: (dict(n=0), dict(reqs=0), dict(n=0, q=0, k=0, v=0, o=0, lse=0, ws=0, nb=0)),
    })


def test_workspace_size():
    lib, nb = L.load(), ctypes.c_int64()

    def call(Hq=8, Hkv=2, dv=128, nodes=4, ctas=152, out=nb):
        return lib.cp_tree_workspace_size(Hq, Hkv, dv, nodes, ctas, out if out is None else ctypes.byref(out))

    refused(call, {BAD: (dict(Hq=0), dict(Hkv=0), dict(Hq=9), dict(Hq=1, Hkv=2), dict(Hq=1 << 21, Hkv=1), dict(nodes=0),
                         dict(ctas=0), dict(ctas=4097), dict(out=None)),
                   KIND: (dict(dv=0), dict(dv=96), dict(dv=256))})
    sizes = []
    for nodes in (1, 4, 32, 33, 2 ** 31 - 1):
        assert call(nodes=nodes) == L.OK and nb.value % 32 == 0
        sizes.append(nb.value)
    assert sizes == sorted(sizes) and sizes[-1] < 1 << 27  # (rows of a unit stop growing)


def test_structures_are_those_of_c(tmp_path):
    """The bytes that the bindings pack lie where C's structures have them."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    assert L.KV_CODES.size == ctypes.sizeof(L.KvCodes)
    kinds = (("cp_rope_args_t", L.ROPE_ARGS, ("q_row_stride", "num_rows", "inverse")),
             ("cp_kv_append_args_t", L.KV_APPEND_ARGS, ("k_row_stride", "num_rows", "x_is_fp32")),
             ("cp_tree_layout_args_t", L.TREE_LAYOUT_ARGS, ("table_stride", "num_reqs", "mask_words")),
             ("cp_attn_tree_args_t", L.ATTN_TREE_ARGS, ("q_row_stride", "num_rows", "scale")))
    body = "".join(f'  printf("%zu", sizeof({c}));\n' + "".join(
        f'  printf(" %zu", offsetof({c}, {f}));\n' for f in fields) + '  printf("\\n");\n' for c, _, fields in kinds)
    src, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "cpattn.h"\nint main(void) {\n' + body + "  return 0;\n}\n")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", cuda, str(src),
                    "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    for line, (name, packed, _) in zip(lines, kinds):
        size, first, ints, last = (int(x) for x in line.split())
        head, rest = packed.format.lstrip("@").split("P")
        longs, tail = rest.split("q")
        assert first == 8 * int(head) and ints == first + 8 * int(longs or 1), name
        assert last == packed.size - 4 and size == -(-packed.size // 8) * 8, name


def test_bindings_refuse_host_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    at, one = torch.zeros(2, dtype=torch.int32), torch.zeros((1, 4), dtype=torch.int32)
    rope = cpa.make_rope([1.0] * 8, device="cpu")
    for call in (lambda: cpa.cp_rope(rope, x, positions=at), lambda: cpa.cp_kv_append((x, x), x, x),
                 lambda: cpa.cp_kv_append(cpa.alloc_kv_cache(4, 2, 64, 64, device="cpu"), x, x),
                 lambda: cpa.cp_tree_layout(at, at[:1], one, 16, 2),
                 lambda: cpa.cp_attn_tree(x, x, x, one, 16, at, at[:1], 0.1)):
        with pytest.raises(ValueError):
            call()


def test_make_rope():
    r = cpa.make_rope(torch.tensor([1.0, 0.5] * 4), axes=[0, 2] * 4, first=16, interleaved=True, device="cpu")
    assert (r.pairs, r.first, r.interleaved, r.axes) == (8, 16, True, 3)
    assert r.table[:, 2].tolist() == [0, 2] * 4
    for bad, err in (([], ValueError), ([[1.0]], ValueError), ([float("nan")], L.CpAttnError), ([1e9], L.CpAttnError)):
        with pytest.raises(err):
            cpa.make_rope(bad, device="cpu")
    with pytest.raises(ValueError):
        cpa.make_rope([1.0] * 8, axes=[0] * 7, device="cpu")
    with pytest.raises(L.CpAttnError):
        cpa.make_rope([1.0] * 8, axes=[8] * 8, device="cpu")
    with pytest.raises(ValueError):
        cpa.Rope(torch.zeros(8, 4))


def test_a_copied_rotation_has_its_own_table():
    r = cpa.make_rope([1.0, 0.5] * 4, first=8, device="cpu")
    for other in (copy.deepcopy(r), pickle.loads(pickle.dumps(r)), copy.copy(r)):
        assert torch.equal(other.table, r.table) and (other.first, other.axes) == (8, 1)
        info = other._of(-1)
        assert info.table == other.table.data_ptr() and (info.pairs, info.first) == (8, 8)
    assert copy.deepcopy(r).table.data_ptr() != r.table.data_ptr()


def test_oracle_rotation():
    """Rotations by two positions add up, the inverse turns back, lengths stay, and scores
    depend on the distance alone."""
    g = np.random.default_rng(0)
    x, y = g.standard_normal((2, 5, 3, 24))
    f = g.uniform(0.001, 1.0, 8)
    at = g.integers(0, 1000, (2, 5))
    axis = [0, 1, 1, 0, 0, 1, 0, 1]
    for inter in (False, True):
        turn = lambda t, p, **kw: op.rotate(t, p, f, axis, first=8, interleaved=inter, **kw)  # noqa: E731
        assert np.allclose(turn(turn(x, at), 3 * at), turn(x, 4 * at), atol=1e-11)
        assert np.allclose(turn(turn(x, at), at, inverse=True), x, atol=1e-12)
        assert np.allclose((turn(x, at) ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.array_equal(turn(x, at)[..., :8], x[..., :8])
        a = (turn(x, at + 100) * turn(y, at + 93)).sum(-1)
        assert np.allclose(a, (turn(x, at + 7) * turn(y, at)).sum(-1), atol=1e-11)


def test_oracle_layout_and_attention():
    slots, positions, seen = op.tree_layout([0, 3, 3, 5], [15, 40, 0], [[4, 2], [0, 1, 3], [5]], 16,
                                            [-1, 0, 0, -1, -1], 6)
    assert slots == [4 * 16 + 15, 2 * 16, 2 * 16 + 1, 80, 81, -1]
    assert positions == [15, 16, 16, 0, 0, 0]
    assert op.mask_words(seen, 1)[:, 0].tolist() == [1, 3, 5, 1, 2]
    # a chain over the whole cache in order is causal attention
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((4, 2, 8)), g.standard_normal((16, 1, 8)), g.standard_normal((16, 1, 8))
    _, _, chain = op.tree_layout([0, 4], [9], [[0]], 16, None, 4)
    got = op.tree_attention(q, k, v, [0, 4], [9], [[0]], 16, chain, 0.5)
    for i in range(4):
        s = 0.5 * np.einsum("hd,nd->hn", q[i], k[:10 + i, 0])
        w = np.exp(s)
        assert np.allclose(got["o"][i], w @ v[:10 + i, 0] / w.sum(-1, keepdims=True))
        assert np.allclose(got["lse"][i], np.log(w.sum(-1)))
