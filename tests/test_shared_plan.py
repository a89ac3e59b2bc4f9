"""The host plan of attention over shared keys: what its counts mean, and how even its
shares are.  No GPU."""

import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L

from test_shared_host import check_plan, read_table


def info(segs, N, Hq=8, Hkv=2):
    t = torch.tensor(segs, dtype=torch.int32).reshape(-1, 8)
    return cpa.make_shared_plan_segs(t, N, Hq, Hkv, num_ctas=152, device="cpu").info


@pytest.mark.parametrize("kv_row0", [-1, 5, 100000, 0x7fffffff])
def test_a_run_that_no_row_sees_lies_anywhere(kv_row0):
    """An empty slot of a padded batch has no key run: where it claims to lie neither counts
    as reached nor refuses the plan."""
    seen = [[0, 3, 99, 0, 0, 100, 0, -1], [0, 1, 0, 1, 100, 1, 0, 0], [2, 1, 3, 1, 101, 4, 0, 2]]
    for empty in ([1, 1, -1, 1, kv_row0, 0, 0, 1], [1, 2, -2, 1, kv_row0, 0, 0, 1],
                  [1, 0, 7, 1, kv_row0, 8, 0, 1]):
        assert info(seen + [empty], 3).kv_rows == 105
        check_plan(seen + [empty], 3, 8, 2, 152)
    assert info([[0, 1, -1, 1, kv_row0, 0, 0, 0]], 1).kv_rows == 0


def test_empty_slots_of_a_padded_batch():
    plan = cpa.make_shared_plan([1, 1, 1, 1], [1, 0, 4, 0], 100, 8, 2, own_row0=[100, -1, 101, 1 << 30],
                                num_ctas=152, device="cpu")
    assert plan.info.kv_rows == 105
    with pytest.raises(L.CpAttnError):  # a slot that holds keys has a place
        cpa.make_shared_plan([1, 1], [1, 1], 100, 8, 2, own_row0=[100, -1], num_ctas=152, device="cpu")


# the planner's costs of a KV tile and of a piece besides, by the kind of its unit
TILE, PIECE = (24, 16, 12), (90, 50, 20)


def kind_of(rows):
    return 0 if rows > 128 else 1 if rows > 8 else 2


def shares(T):
    """The cost of each block's list; a single unit's keys that were cut between the block's
    two streams are one piece."""
    out = []
    for c in T["ctas"]:
        cost, last = 0, None
        for name in ("dual", "single", "small"):
            end = c["single2" if name == "single" else name + "1"]
            for p in T["pieces"][c[name + "0"]: end]:
                kind = kind_of(p["rows"])
                on = kind == 1 and last is not None and p["key0"] == last["key0"] + last["keys"] and \
                    all(p[x] == last[x] for x in ("q_row0", "r0", "rows", "kv_head"))
                cost += TILE[kind] * ((p["keys"] + 127) // 128) + (0 if on else PIECE[kind])
                last = p
        out.append(cost)
    return out


BATCHES = {
    # name: Hq, Hkv, q_lens, own_lens, prefix
    "decode": (32, 8, [1] * 64, [37 * i % 2048 + 1 for i in range(64)], 65536),
    "past_a_tile": (32, 8, [1] * 65, [1] * 65, 65536),
    "one": (32, 8, [1], [100], 1024),
    "verify": (32, 8, [1 + 3 * i % 8 for i in range(16)], [20 + 61 * i % 1000 for i in range(16)], 16383),
    "aligned_tiles": (32, 8, [1] * 256, [37 * i % 2048 + 1 for i in range(256)], 65536),
    "single": (8, 8, [90, 30], [4000, 700], 20000),
    "chunk": (32, 8, [700, 9], [1500, 9], 5000),
    "small": (8, 8, [1] * 300, [11 * i % 900 + 1 for i in range(300)], 0),
}


@pytest.mark.parametrize("num_ctas", [152, 40])
@pytest.mark.parametrize("name", sorted(BATCHES))
def test_shares_are_near_the_average(name, num_ctas):
    """The largest share of these batches is within one piece and one tile of the average, no
    share exceeds the budget, and the budget has a bound.  It is the smallest that fits: with one less, every block is filled until
    the next piece's fixed part and a tile do not go in (the last block before the small
    units and the one before each aligned tile may hold less), and work is left over; and
    the blocks' ends cut at most num_ctas pieces more than there are units."""
    Hq, Hkv, q_lens, own, prefix = BATCHES[name]
    segs = cpa.shared_segments(q_lens, own, prefix)
    plan = cpa.make_shared_plan_segs(segs, sum(q_lens), Hq, Hkv, num_ctas=num_ctas, device="cpu")
    T = read_table(plan)
    cost, budget = shares(T), plan.info.budget
    assert max(cost) <= budget
    tiles = units = worst = aligned = 0
    for q_row0, q_len, pos0, step, _, _, _, _ in segs.tolist():
        packed = q_len * Hq // Hkv
        for r0 in range(0, packed, 256):
            rows = min(256, packed - r0)
            keys = max(0, pos0 + (r0 + rows - 1) // (Hq // Hkv) * step + 1)
            kind, n = kind_of(rows), (keys + 127) // 128
            if n == 0:
                continue
            worst = max(worst, TILE[kind] + PIECE[kind])
            tiles += Hkv * n * TILE[kind]
            units += Hkv * PIECE[kind]
            aligned += kind == 0 and r0 > 0 and Hkv * n * TILE[0] // 8 >= budget - 1
    assert max(cost) <= sum(cost) / num_ctas + worst
    most = tiles + units + num_ctas * max(PIECE[k] for k in range(3) if TILE[k] + PIECE[k] <= worst)
    assert budget - 1 <= worst + most / (num_ctas - 1 - aligned), (budget, worst, most)
