"""Host side of the quantised cache and of attention over shared keys: the plan
covers every (row, head, key) once, its shares are even, and bad arguments are
refused before anything is launched.  No GPU."""

import ctypes
import random

import numpy as np
import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L
from oracle import shared as osh

ROWS = 256  # CPATTN_SHARED_ROWS
CTA = ("dual0", "dual1", "single0", "single1", "single2", "small0", "small1", "u0")
PIECE = ("q_row0", "q_pos0", "q_pos_step", "r0", "rows", "kv_head", "kv_row", "key0", "keys",
         "ws_row", "u0", "u1")
UNIT = ("ws_row", "parts", "rows", "u0")


def read_table(plan):
    i, t = plan.info, plan.table.tolist()
    at, out = 0, {}
    for name, n, fields in (("ctas", i.num_ctas, CTA), ("pieces", i.num_pieces, PIECE),
                            ("units", i.num_units, UNIT)):
        out[name] = [dict(zip(fields, t[at + len(fields) * j: at + len(fields) * (j + 1)]))
                     for j in range(n)]
        at += n * len(fields)
    for name, n in (("row_first", i.num_q_rows + 1), ("entries", 2 * i.num_entries)):
        at += at % 2 if name == "entries" else 0
        out[name] = t[at: at + n]
        at += n
    assert at == len(t) == i.table_ints
    return out


def tiles_of(pieces):
    return sum((p["keys"] + 127) // 128 for p in pieces)


def check_plan(segs, N, Hq, Hkv, num_ctas):
    plan = cpa.make_shared_plan_segs(torch.tensor(segs, dtype=torch.int32).reshape(-1, 8), N, Hq,
                                     Hkv, num_ctas=num_ctas, device="cpu")
    T, g = read_table(plan), Hq // Hkv
    # each piece belongs to one block; dual pieces first, small ones last and in blocks of
    # their own; the streams' tiles are even
    kinds = [0 if p["rows"] > 128 else 1 if p["rows"] > 8 else 2 for p in T["pieces"]]
    assert kinds == sorted(kinds)
    at = [0, kinds.count(0), kinds.count(0) + kinds.count(1)]
    ends = at[1:] + [len(kinds)]
    for c in T["ctas"]:
        assert [c["dual0"], c["single0"], c["small0"]] == at
        assert c["dual0"] <= c["dual1"] and c["single0"] <= c["single1"] <= c["single2"]
        at = [c["dual1"], c["single2"], c["small1"]]
        assert c["small0"] == c["small1"] or (c["dual0"] == c["dual1"] and
                                              c["single0"] == c["single2"])
        two = [tiles_of(T["pieces"][a:b]) for a, b in ((c["single0"], c["single1"]),
                                                       (c["single1"], c["single2"]))]
        assert two[0] - two[1] in (0, 1)
    assert at == ends
    # partial rows do not overlap and fill the workspace
    used = np.zeros(plan.info.ws_rows, dtype=np.int32)
    for p in T["pieces"]:
        assert 1 <= p["rows"] <= ROWS and p["keys"] >= 1
        parts = p["rows"]
        assert 0 <= p["ws_row"] and p["ws_row"] + parts <= plan.info.ws_rows
        used[p["ws_row"]: p["ws_row"] + parts] += 1
        assert p["kv_row"] + p["keys"] <= plan.info.kv_rows
    assert (used == 1).all()
    # every row's entries lead to pieces that cover its runs' keys once
    ends = {p["ws_row"]: p for p in T["pieces"]}
    for n, runs in enumerate(osh.row_runs(segs, N)):
        e0, e1 = T["row_first"][n], T["row_first"][n + 1]
        assert e1 - e0 == len(runs)
        for h in range(Hq):
            for e, (kv0, seen) in zip(range(e0, e1), runs):
                unit0, i = T["entries"][2 * e], T["entries"][2 * e + 1]
                packed = i * g + h % g
                u = T["units"][unit0 + packed // ROWS * Hkv + h // g]
                at, part = 0, 0
                while part < u["parts"]:
                    p = ends[u["ws_row"] + part * u["rows"]]
                    assert p["kv_head"] == h // g and p["r0"] == packed // ROWS * ROWS
                    assert p["q_row0"] + (p["r0"] + packed % ROWS) // g == n
                    assert packed % ROWS < p["rows"] == u["rows"]
                    assert p["key0"] == at and p["kv_row"] == kv0 + at
                    at += p["keys"]
                    part += 1
                assert part == u["parts"] and at >= seen
    return plan, T


@pytest.mark.parametrize("seed", range(24))
def test_plan_covers_every_key_once(seed):
    rng = random.Random(seed)
    Hq, Hkv = rng.choice([(8, 8), (8, 2), (12, 4), (7, 1), (32, 1)])
    B = rng.choice([1, 2, 5, 9])
    q_lens = [rng.randint(0, rng.choice([1, 1, 4, 90])) for _ in range(B)]
    own = [rng.choice([0, n, n + rng.randint(0, 700), max(0, n - 2)]) for n in q_lens]
    prefix = rng.choice([0, 1, 127, 128, 129, rng.randint(1, 3000)])
    segs = cpa.shared_segments(q_lens, own, prefix, prefix_row0=rng.randint(0, 5)).tolist()
    if seed % 3 == 0 and sum(q_lens) > 2:  # a nested prefix over part of the batch
        segs.insert(1, [1, sum(q_lens) - 2, 299, 0, 7, 300, 0, -1])
    check_plan(segs, sum(q_lens), Hq, Hkv, rng.choice([2, 3, 16, 152]))


def test_plan_empty_batches():
    for segs, N in (([], 0), ([], 3), ([[0, 0, 5, 1, 0, 6, 0, 0]], 2),
                    ([[0, 2, -4, 1, 0, 0, 0, 0]], 2)):
        plan, T = check_plan(segs, N, 8, 2, 152)
        assert plan.info.num_pieces == 0


def test_plan_shares_are_even():
    """64 queries on a 64K prefix with ragged own keys over 152 blocks: the
    largest share is within one tile and two pieces of the average, a KV tile of
    more than 128 packed rows counted as 1.5."""
    rng = random.Random(5)
    own = [rng.randint(1, 2048) for _ in range(64)]
    segs = cpa.shared_segments([1] * 64, own, 65536).tolist()
    _, T = check_plan(segs, 64, 32, 8, 152)
    for kind in ("dual", "small"):
        cost = [tiles_of(T["pieces"][c[kind + "0"]:c[kind + "1"]]) + c[kind + "1"] - c[kind + "0"]
                for c in T["ctas"]]
        cost = [x for x in cost if x]
        assert len(cost) > 20 and sorted(cost)[-1] <= sum(cost) / len(cost) + 8


def seg_ptr(rows):
    t = torch.tensor(rows, dtype=torch.int32).reshape(-1, 8)
    return t, ctypes.c_void_p(t.data_ptr())


def test_plan_refusals():
    lib, info = L.load(), L.SharedPlanInfo()

    def size(rows, N=4, Hq=8, Hkv=2, ctas=152, n=None, out=info):
        t, p = seg_ptr(rows)
        return lib.cp_shared_plan_size(p, t.shape[0] if n is None else n, N, Hq, Hkv, ctas, out)

    good = [0, 4, 9, 0, 0, 10, 0, 0]
    assert size([good]) == L.OK
    for bad in ([0, 5, 9, 0, 0, 10, 0, 0], [1, 4, 9, 0, 0, 10, 0, 0], [-1, 2, 9, 0, 0, 10, 0, 0],
                [0, -1, 9, 0, 0, 10, 0, 0], [0, 4, 9, -1, 0, 10, 0, 0], [0, 4, 9, 0, -1, 10, 0, 0],
                [0, 4, 9, 1, 0, 10, 0, 0], [0, 4, -9, 0, 0, -1, 0, 0]):
        assert size([bad]) == L.ERR_INVALID_ARG, bad
    assert size([[0, 4, 9, 0, 0x7fffffff, 10, 0, 0]]) == L.ERR_TOO_LARGE
    assert size([good], Hq=6, Hkv=4) == L.ERR_INVALID_ARG
    assert size([good], Hkv=0) == L.ERR_INVALID_ARG
    assert size([good], ctas=0) == L.ERR_INVALID_ARG
    assert size([good], ctas=1) == L.ERR_INVALID_ARG
    assert size([good], ctas=4097) == L.ERR_INVALID_ARG
    assert size([good], N=-1) == L.ERR_INVALID_ARG
    assert size([good], n=-1) == L.ERR_INVALID_ARG
    assert size([good], out=None) == L.ERR_INVALID_ARG
    assert lib.cp_shared_plan_size(None, 1, 4, 8, 2, 152, info) == L.ERR_INVALID_ARG
    # the second pass takes only the table that was sized
    assert size([good]) == L.OK
    t, p = seg_ptr([good])
    table = torch.full((info.table_ints,), -7, dtype=torch.int32)
    tp = ctypes.c_void_p(table.data_ptr())
    other, op = seg_ptr([[0, 4, 999, 0, 0, 1000, 0, 0]])
    assert lib.cp_shared_plan(op, 1, info, tp) == L.ERR_INVALID_ARG
    assert lib.cp_shared_plan(p, 0, info, tp) == L.ERR_INVALID_ARG
    info.table_ints -= 1
    assert lib.cp_shared_plan(p, 1, info, tp) == L.ERR_INVALID_ARG
    info.table_ints += 1
    assert (table == -7).all()
    assert lib.cp_shared_plan(p, 1, info, tp) == L.OK
    nbytes = ctypes.c_int64()
    for dv in (0, 6, 1028):
        assert lib.cp_shared_workspace_size(info, dv, ctypes.byref(nbytes)) == L.ERR_INVALID_ARG
    assert lib.cp_shared_workspace_size(info, 128, ctypes.byref(nbytes)) == L.OK
    assert nbytes.value >= 16
    with pytest.raises(ValueError):
        cpa.shared_segments([1, 1], [1], 4)
    with pytest.raises(ValueError):
        cpa.shared_segments([1], [-1], 4)
    with pytest.raises(ValueError):
        cpa.shared_segments([1, 1], [1, 1], 4, own_row0=[0])
    with pytest.raises(ValueError):
        cpa.make_shared_plan_segs(torch.zeros(3, 7, dtype=torch.int32), 3, 8, 2, num_ctas=1,
                                  device="cpu")


def test_attention_refusals():
    """Every call fails its checks before any launch (pointers are never used)."""
    lib = L.load()
    plan = cpa.make_shared_plan([1, 1], [5, 9], 100, 8, 2, num_ctas=152, device="cpu")
    nbytes = cpa.cp_shared_workspace_size(plan, 128)
    P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(9)]
    base = dict(plan=plan.info, table=P[0], q=P[1], qr=1024, qh=128, k=P[2], kr=256, kh=128,
                ks=None, v=P[3], vr=256, vh=128, vs=None, ss=0, rows=114, d=128, dv=128, scale=0.1,
                o=P[4], f32=0, lse=P[5], ws=P[6], nb=nbytes, status=None, stream=None)

    def call(**kw):
        return lib.cp_attn_shared(*{**base, **kw}.values())

    off = ctypes.c_void_p(0x10008)
    for kw in (dict(plan=None), dict(table=None), dict(q=None), dict(k=None), dict(v=None),
               dict(o=None), dict(lse=None), dict(ws=None), dict(nb=nbytes - 1), dict(rows=113),
               dict(rows=-1), dict(scale=0.0), dict(scale=float("nan")), dict(ks=P[7]),
               dict(vs=P[7]), dict(kr=248), dict(kh=120), dict(vr=248), dict(vh=64), dict(qr=-8),
               dict(ks=P[7], vs=P[8], ss=113)):
        assert call(**kw) == L.ERR_INVALID_ARG, kw
    for kw in (dict(d=64), dict(dv=64), dict(d=96, dv=96), dict(d=576, dv=512)):
        assert call(**kw) == L.ERR_UNSUPPORTED, kw
    for kw in (dict(table=off), dict(q=off), dict(k=off), dict(v=off), dict(o=off), dict(ws=off),
               dict(lse=ctypes.c_void_p(0x10002)), dict(qr=1028), dict(qh=132), dict(kr=260),
               dict(vh=132), dict(ks=P[7], vs=P[8], ss=200, kr=264),
               dict(ks=ctypes.c_void_p(0x10001), vs=P[8], ss=200)):
        assert call(**kw) == L.ERR_ALIGNMENT, kw
    bad = L.SharedPlanInfo.from_buffer_copy(plan.info)
    bad.num_pieces += 1
    assert call(plan=bad) == L.ERR_INVALID_ARG
    # a batch without rows does nothing
    none = cpa.make_shared_plan([], [], 100, 8, 2, num_ctas=152, device="cpu")
    assert call(plan=none.info, q=None, o=None, lse=None, ws=None, nb=0) == L.OK


def test_cache_refusals():
    lib = L.load()
    P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(9)]
    C = lambda **kw: L.KvCodes(**{**dict(codes=0x50000, scales=0x60000, row_stride=256,  # noqa: E731
                                         head_stride=128, scale_stride=64), **kw})
    qbase = dict(k=P[0], kr=256, kh=128, v=P[1], vr=256, vh=128, f32=0, n=4, H=2, d=128, dv=128,
                 slots=P[2], kc=C(), vc=C(), rows=64, status=None, stream=None)

    def quant(**kw):
        return lib.cp_kv_quantize(*{**qbase, **kw}.values())

    for kw in (dict(n=-1), dict(rows=-1), dict(H=0), dict(kc=None), dict(vc=None), dict(v=None),
               dict(k=None), dict(kr=-8), dict(vh=-8), dict(kc=C(codes=None)),
               dict(vc=C(scales=None)), dict(kc=C(head_stride=112)), dict(kc=C(row_stride=240)),
               dict(kc=C(scale_stride=63)), dict(rows=65)):
        assert quant(**kw) == L.ERR_INVALID_ARG, kw
    for kw in (dict(d=120), dict(d=8), dict(d=1040), dict(dv=0), dict(dv=100)):
        assert quant(**kw) == L.ERR_UNSUPPORTED, kw
    for kw in (dict(k=ctypes.c_void_p(0x10008)), dict(slots=ctypes.c_void_p(0x10002)),
               dict(kr=260), dict(vh=132), dict(f32=1, kh=130), dict(kc=C(codes=0x50008)),
               dict(vc=C(scales=0x60002)), dict(kc=C(row_stride=264))):
        assert quant(**kw) == L.ERR_ALIGNMENT, kw
    assert quant(n=0, k=None, v=None) == L.OK

    dbase = dict(kc=C(), vc=C(), rows=64, H=2, d=128, dv=128, idx=P[0], n=4, ko=P[1], vo=P[2],
                 f32=0, status=None, stream=None)

    def deq(**kw):
        return lib.cp_kv_dequantize(*{**dbase, **kw}.values())

    for kw in (dict(n=-1), dict(rows=-1), dict(H=0), dict(kc=None), dict(vc=None), dict(ko=None),
               dict(vo=None), dict(kc=C(scale_stride=10))):
        assert deq(**kw) == L.ERR_INVALID_ARG, kw
    assert deq(d=24) == L.ERR_UNSUPPORTED
    for kw in (dict(ko=ctypes.c_void_p(0x10004)), dict(idx=ctypes.c_void_p(0x10001))):
        assert deq(**kw) == L.ERR_ALIGNMENT, kw
    assert deq(n=0, ko=None, vo=None) == L.OK


def test_bindings_refuse_host_tensors():
    cache = cpa.alloc_kv_cache(4, 2, 64, 64, device="cpu")
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        cpa.cp_kv_quantize(cache, x, x)
    with pytest.raises(ValueError):
        cpa.cp_kv_dequantize(cache)
    plan = cpa.make_shared_plan([1], [4], 0, 2, 2, num_ctas=152, device="cpu")
    with pytest.raises(ValueError):
        cpa.cp_attn_shared(plan, x[:1], x, x, 0.1)


def test_oracle_codes():
    """The oracle's e4m3 against torch's conversion on every code and the midpoints
    between neighbours (ties), and its exponent against 448 times powers of two."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    fin = np.unique(codes[np.isfinite(codes)].astype(np.float64))
    mids = (fin[1:] + fin[:-1]) / 2
    for y in (fin, mids, np.nextafter(mids, 1e9), np.nextafter(mids, -1e9)):
        y32 = y.astype(np.float32).astype(np.float64)
        want = torch.tensor(y32, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
        assert (osh.e4m3(y32) == want).all()
    for e in (-117, -3, 0, 7, 119):
        a = 448.0 * 2.0 ** e
        assert osh.scale_exponents(np.array([[a]]))[0] == e
        up = np.nextafter(a, np.inf)
        assert osh.scale_exponents(np.array([[up]]))[0] == min(119, e + 1)
    assert osh.scale_exponents(np.zeros((1, 4)))[0] == -117
    assert osh.scale_exponents(np.array([[np.inf, 448.0, np.nan]]))[0] == 0
