"""cos and sin of small angles, and next to a quarter turn, keep fp32's relative bits.

A pair (1, 0) becomes (cos t, sin t).  The angle is off by at most |p| 2^-64 turns; its rest of a
quarter turn is rounded to fp32 twice, 2^-23 of the rest, by which a sine moves at most in proportion
and a cosine by pi / 4 of that; the functions are off by 2 units in the last place (2^-22 of the value at
most) and the product by 2^-24: together 7 2^-24 of the value, below 2^-21, and 2 pi |p| 2^-64."""

import numpy as np
import pytest
import torch

import context_causal_attention_cp_gb300 as cpa
from oracle import paged as op

from test_gpu_shared import f64

pytestmark = pytest.mark.gpu

SLOW = [1e-9, 4.5e-6, 3e-7, 2.0 ** -31, 1e-11, 500000.0 ** (-63 / 64), -2e-8, 1e-4]
NEAR = [np.pi / 2 - 1e-7, np.pi - 3e-8, 1.5 * np.pi + 1e-6, 2 * np.pi + 2e-9, -np.pi / 2 + 1e-8, np.pi / 4, 0.3, -np.pi + 1e-5]


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("freqs,positions", [(SLOW, [0, 1, -1, 2, 7, 100, 4097, -65536]), (NEAR, [1, -1, 2])],
                         ids=["slow", "near"])
def test_small_sines_and_cosines(freqs, positions, interleaved):
    pos = np.array([positions])
    rope = cpa.make_rope(freqs, interleaved=interleaved)
    x = torch.zeros((len(positions), 1, 16), device="cuda")
    x[:, :, ::2] = 1.0
    if not interleaved:
        x = torch.cat([torch.ones_like(x[..., :8]), torch.zeros_like(x[..., 8:])], -1)
    for inverse in (False, True):
        y, _ = cpa.cp_rope(rope, x, positions=torch.tensor(positions, dtype=torch.int32, device="cuda"), inverse=inverse)
        want = op.rotate(f64(x), pos, freqs, interleaved=interleaved, inverse=inverse)
        # (the oracle's own: an angle of up to 16 in a double, and its cos or sin; near p f = pi / 2 also pi's)
        tol = 2.0 ** -21 * np.abs(want) + 2 * np.pi * np.abs(pos).T[:, :, None] * 2.0 ** -64 + 2.0 ** -48
        if freqs is SLOW:  # (angles below 1: a double's 2^-53 of each sine)
            tol = 2.0 ** -21 * np.abs(want) + 2 * np.pi * np.abs(pos).T[:, :, None] * 2.0 ** -64
        off = np.abs(f64(y) - want)
        assert (off <= tol).all(), f"{(off / np.maximum(tol, 1e-300)).max():.1f} of the tolerance"
