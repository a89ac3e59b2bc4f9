"""The host plan of attention over shared keys: what its counts mean, and how even its
shares are.  No GPU."""

import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from context_causal_attention_cp_gb300 import _lib as L

from test_shared_host import check_plan


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
