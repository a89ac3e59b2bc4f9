"""make_rope's frequencies keep their 64 bits, however they are given.  No GPU."""

import numpy as np
import pytest
import torch

import context_causal_attention_cp_gb300 as cpa

FREQS = [500000.0 ** (-c / 16) for c in range(16)]


@pytest.mark.parametrize("given", [list, tuple, np.array, lambda f: torch.tensor(f, dtype=torch.float64),
                                   lambda f: [np.float64(x) for x in f]],
                         ids=["list", "tuple", "array", "tensor", "list of float64"])
def test_frequencies_keep_64_bits(given):
    table = cpa.make_rope(given(FREQS), device="cpu").table.numpy()
    F = table[:, 0].view(np.uint32).astype(object) | table[:, 1].view(np.uint32).astype(object) << 32
    for f, got in zip(FREQS, F):
        # f / 2 pi in a double: 2 roundings and that of 2 pi, 2^-53 each; the table counts in steps of
        # 2^-64 turns, half of which is 2^-65
        assert abs(int(got) / 2.0 ** 64 - f / (2 * np.pi)) <= 2.0 ** -51 * f + 2.0 ** -65, f


def test_frequencies_in_32_bits_are_taken_as_they_are():
    f = torch.tensor(FREQS)
    assert torch.equal(cpa.make_rope(f, device="cpu").table, cpa.make_rope(f.double(), device="cpu").table)
    assert torch.equal(cpa.make_rope([1, 0] * 4, device="cpu").table, cpa.make_rope([1.0, 0.0] * 4, device="cpu").table)
