"""Copies of the plan of the shared-key attention and of the quantised cache: a copy works
from its own tensors, not from the memory of the first one's."""

import copy
import ctypes
import dataclasses
import pickle

import pytest
import torch

import context_causal_attention_cp_gb300 as cpa


def addresses(x):
    """The integers that x is made of, those of a ctypes structure among them."""
    if isinstance(x, ctypes.Structure):
        x = tuple(getattr(x, n) for n, _ in x._fields_)
    return [n for y in x for n in addresses(y)] if isinstance(x, tuple) else [x]


def test_copies_hold_no_address_of_the_first():
    plan = cpa.make_shared_plan([1], [4], 0, 2, 2, num_ctas=152, device="cpu")
    cache = cpa.alloc_kv_cache(4, 2, 64, 64, device="cpu")
    copies = [(x, y) for x in (plan, cache) for y in (copy.deepcopy(x), copy.deepcopy(copy.copy(x)))]
    copies.append((plan, pickle.loads(pickle.dumps(plan))))
    for first, other in copies:
        names = [f.name for f in dataclasses.fields(first)]
        tensors = {n: getattr(first, n) for n in names if isinstance(getattr(first, n), torch.Tensor)}
        assert not {t.data_ptr() for t in tensors.values()} & set(addresses(tuple(vars(other).values())))
        for n, t in tensors.items():
            o = getattr(other, n)
            assert (o.shape, o.stride(), o.dtype) == (t.shape, t.stride(), t.dtype)


@pytest.mark.gpu
def test_copies_of_a_plan_and_a_cache_use_their_own_memory():
    """copy.deepcopy and dataclasses.replace give objects that work from their own tensors."""
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(s, generator=g, device="cuda").bfloat16()
               for s in ((4, 8, 128), (500, 2, 128), (500, 2, 128)))
    plan = cpa.make_shared_plan([1] * 4, [10] * 4, 300, 8, 2)
    cache = cpa.alloc_kv_cache(500, 2, 128, 128)
    cpa.cp_kv_quantize(cache, k, v)
    kw = dict(k_scale=cache.k_scale, v_scale=cache.v_scale)
    o, lse, _ = cpa.cp_attn_shared(plan, q, cache.k, cache.v, 0.1, **kw)
    rows = cpa.cp_kv_dequantize(cache)
    plans = [copy.deepcopy(plan), dataclasses.replace(plan, table=plan.table.clone())]
    caches = [copy.deepcopy(cache), dataclasses.replace(cache, k=cache.k.clone(), v=cache.v.clone())]
    plan.table.zero_()  # the lists of all blocks empty
    cache.k.view(torch.uint8).zero_()
    cache.v.view(torch.uint8).zero_()
    for p, c in zip(plans, caches):
        o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
        cpa.cp_attn_shared(p, q, c.k, c.v, 0.1, k_scale=c.k_scale, v_scale=c.v_scale, out=o2, lse=lse2)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        for a, b in zip(cpa.cp_kv_dequantize(c), rows):
            assert torch.equal(a, b)
    # a tensor that was given other memory of the same layout
    cache.k.data, plan.table.data = caches[0].k.clone(), plans[0].table.clone()
    assert torch.equal(cpa.cp_kv_dequantize(cache)[0], rows[0])
    o2, _, _ = cpa.cp_attn_shared(plan, q, caches[0].k, caches[0].v, 0.1, **kw)
    assert torch.equal(o2, o)
