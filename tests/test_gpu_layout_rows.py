"""Every row of a layout is written, whatever q_start holds: rows of no request have slot -1, so that
an append that follows writes nothing for them."""

import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L

from test_gpu_guards import Guarded
from test_gpu_tree import i32

pytestmark = pytest.mark.gpu

N, PAGE = 200, 16
STARTS = [[0, 250, 200], [0, -4, 200], [7, 60, 200], [0, 60, 2 ** 31 - 1], [0, 60, -2 ** 31], [-5, 60, 200], [0, 120, 60],
          [300, 250, 220], [-1, -2, -3], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]]


@pytest.mark.parametrize("tree", [True, False], ids=["tree", "chain"])
@pytest.mark.parametrize("starts", STARTS, ids=str)
def test_every_row_is_written(starts, tree):
    table, lens = i32([list(range(20)), list(range(20, 40))]), [30, 9]
    parents = i32([-1] * N) if tree else None
    outs = [Guarded((N,), torch.int32, 55), Guarded((N,), torch.int32, -55), Guarded((N, 7), torch.int32, 55)]
    status = cpa.new_status()
    slots, positions, mask = cpa.cp_tree_layout(i32(starts), i32(lens), table, PAGE, N, parents=parents, slots=outs[0].t,
                                                positions=outs[1].t, mask=outs[2].t if tree else None, status=status)
    for g in outs:
        g.check(str(starts))
    assert int(status.item()) == L.ERR_RANGE
    # a row is one of no request, or of one that is right by itself
    mine = [{-1} for _ in range(N)]
    for b, (s0, s1) in enumerate(zip(starts, starts[1:])):
        if 0 <= s0 <= s1 <= N and not (b == 0 and s0):
            for i in range(s1 - s0):
                mine[s0 + i].add(PAGE * 20 * b + lens[b] + i)
    assert all(x in y for x, y in zip(slots.tolist(), mine))
    assert (positions >= 0).all()
    assert not tree or not (mask == 55).any()


def test_rows_of_no_request_are_not_appended():
    for starts in STARTS[:3] + STARTS[5:6]:
        slots = torch.full((N,), 3, dtype=torch.int32, device="cuda")  # (of an earlier step, say)
        cpa.cp_tree_layout(i32(starts), i32([30, 9]), i32([list(range(20)), list(range(20, 40))]), PAGE, N, slots=slots)
        cache = (torch.zeros((640, 1, 64), dtype=torch.bfloat16, device="cuda"), None)
        cpa.cp_kv_append(cache, torch.ones((N, 1, 64), dtype=torch.bfloat16, device="cuda"), None, slots)
        assert not cache[0][:9].any()
