"""Outputs of a rotation beside their input in one buffer: taken when no element of one lies on the
other, refused else.  Each call has a K at an odd address, which is refused behind Q's places, so
that nothing is launched.  No GPU."""

import itertools

import pytest

from context_causal_attention_cp_gb300 import _lib as L

BASE = 1 << 20


def call(q, qo, n, Hq, d, qr, qh, qor, qoh):
    a = dict(q=q, k=4, qo=qo, ko=4, at=0x800000, status=0, qr=qr, qh=qh, kr=256, kh=128, qor=qor, qoh=qoh, kor=256,
             koh=128, axis=0, n=n, Hq=Hq, Hk=1, d=d, f32=0, inverse=0)
    rope = L.RopeInfo(table=0x900000, pairs=8, first=0, interleaved=0, axes=1)
    rc = L.load().cp_rope(rope, L.ROPE_ARGS.pack(*a.values()), None)
    assert rc in (L.ERR_ALIGNMENT, L.ERR_INVALID_ARG)
    return rc == L.ERR_ALIGNMENT  # (K's, so Q's places were taken)


def cells(at, n, H, d, row, head):
    return {at // 2 + i * row + j * head + c for i in range(n) for j in range(H) for c in range(0, d, 8)}


def test_slots_of_one_buffer():
    n, H, d = 5, 4, 64
    for slots in (2, 3):
        row, head = H * slots * d, slots * d
        for a, b in itertools.product(range(slots), repeat=2):
            assert call(BASE + 2 * a * d, BASE + 2 * b * d, n, H, d, row, head, row, head), (slots, a, b)
    # by heads before rows
    row, head = 2 * d, n * 2 * d
    assert call(BASE, BASE + 2 * d, n, H, d, row, head, row, head)
    # one row, one head
    assert call(BASE, BASE + 2 * d, 1, H, d, 0, 2 * d, 0, 2 * d)
    assert call(BASE, BASE + 2 * d, n, 1, d, 2 * d, 0, 2 * d, 0)


def test_rows_side_by_side_with_heads_of_other_strides():
    n, H, d = 5, 3, 64
    assert call(BASE, BASE + 2 * 200, n, H, d, 640, 64, 640, 128)
    assert call(BASE + 2 * 384, BASE, n, H, d, 640, 96, 640, 64)
    assert not call(BASE, BASE + 2 * 184, n, H, d, 640, 64, 640, 128)
    assert not call(BASE, BASE + 2 * 64, n, H, d, 640, 128, 640, 192)


@pytest.mark.parametrize("n,H,row,head", [(3, 4, 512, 128), (4, 3, 64, 512), (2, 5, 1024, 64), (6, 1, 192, 64), (1, 6, 64, 160),
                                          (5, 2, 208, 80), (3, 3, 432, 128)])
def test_taken_exactly_when_nothing_meets(n, H, row, head):
    d = 64
    for off in range(-row * n - 256, row * n + 256, 8):
        x, y = cells(BASE, n, H, d, row, head), cells(BASE + 2 * off, n, H, d, row, head)
        # (places are multiples of 8 elements)
        assert call(BASE, BASE + 2 * off, n, H, d, row, head, row, head) == (off == 0 or not x & y), off
