"""Which layouts of x and y dsa_rope takes, decided on the host before anything
touches a device.  Every call here passes positions that are not aligned to
their elements: a layout that would be taken is answered with
DSA_ERR_MISALIGNED, and nothing is launched."""
import ctypes as C
import itertools

import pytest

import dsa_sparse_attention_score_gb300 as dsa
from dsa_sparse_attention_score_gb300 import build as dsa_build

X = 1 << 40                                            # never dereferenced
P = C.c_void_p


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


def taken(L, T, H, D, xt, xh, yt, yh, gap, dt=2, rot=2):
    """Is y, `gap` values behind x, taken?"""
    r = dsa.dsa_rope_t(0x8000, rot, 1, 1.0)
    code = L.dsa_rope(P(X), xt, xh, P(X + gap * (4 if dt == 0 else 2)), yt, yh, dt, T, H, D, 0, P(0x40002), C.byref(r), 0, None)
    assert code in (dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_MISALIGNED), code
    return code == dsa.DSA_ERR_MISALIGNED


def cells(T, H, D, st, sh, at=0):
    return [at + t * st + h * sh + i for t in range(T) for h in range(H) for i in range(D)]


def test_slices_whose_next_token_is_the_others_last_head(L):
    # x[0, 1] and y[1, 0] are both the values 192 .. 255, whichever comes first
    assert not taken(L, 2, 2, 64, 192, 128, 192, 128, -64)
    assert not taken(L, 2, 2, 64, 192, 128, 192, 128, 64)
    # the same with heads outside tokens
    assert not taken(L, 2, 2, 64, 128, 192, 128, 192, -64)
    assert not taken(L, 2, 2, 64, 128, 192, 128, 192, 64)


def test_slices_packed_tightly_are_taken(L):
    for gap in (64, -64):
        assert taken(L, 2, 2, 64, 256, 128, 256, 128, gap)           # [T, H, x | y]
        assert taken(L, 2, 2, 64, 128, 256, 128, 256, gap)           # [H, T, x | y]
        assert taken(L, 1, 5, 64, 0, 128, 0, 128, gap)
        assert taken(L, 5, 1, 64, 128, 0, 128, 0, gap)
        assert not taken(L, 2, 2, 64, 255, 128, 255, 128, gap)
        assert not taken(L, 2, 2, 64, 256, 127, 256, 127, gap)
    # groups of heads of one buffer: [T, heads of x | heads of y, D]
    assert taken(L, 7, 4, 64, 8 * 64, 64, 8 * 64, 64, 4 * 64)
    assert taken(L, 7, 4, 64, 8 * 64, 64, 8 * 64, 64, -4 * 64)
    assert not taken(L, 7, 4, 64, 8 * 64, 64, 8 * 64, 64, 3 * 64)
    assert not taken(L, 7, 4, 64, 7 * 64, 64, 7 * 64, 64, 4 * 64)


def test_what_is_taken_shares_nothing(L):
    """Every small layout: rows of y apart from one another, and x and y the
    same rows or no value of either in the other."""
    n = 0
    for T, H, D in itertools.product((1, 2, 3), (1, 2, 3), (2, 3)):
        for st, sh in itertools.product((0, 2, 3, 4, 5, 6, 8, 9, 12, 16), repeat=2):
            for other in ((st, sh), (sh, st), (st + 1, sh)):
                for gap in (0, 1, 2, 3, 4, 5, 6, 9, -1, -2, -3, -4, -7, -10):
                    if not taken(L, T, H, D, *other, st, sh, gap):
                        continue
                    n += 1
                    y = cells(T, H, D, st, sh, gap)
                    assert len(set(y)) == len(y), (T, H, D, st, sh)
                    x = cells(T, H, D, *other)
                    assert x == y or not set(x) & set(y), (T, H, D, other, st, sh, gap)
    assert n > 500


def test_strides_as_far_as_a_head_major_view_has_them(L):
    # [H, T, D] passed as [T, H, D]: head stride T * D
    assert taken(L, 131072, 32, 128, 128, 131072 * 128, 128, 131072 * 128, 32 * 131072 * 128)
    assert taken(L, 131072, 32, 128, 128, 131072 * 128, 128, 131072 * 128, 0)
    assert taken(L, 1 << 20, 8, 64, 8 * 64, 64, 64, 64 << 20, 1 << 34)
    # an axis may reach over 2^40 values, no further
    far = 1 << 40
    assert taken(L, 4, 2, 64, 64, far // 2, 64, 256, 1 << 42) and not taken(L, 4, 2, 64, 64, far // 2 + 1, 64, 256, 1 << 42)
    assert taken(L, 4, 2, 64, 64, 256, 64, far // 2, 1 << 42) and not taken(L, 4, 2, 64, 64, 256, 64, far // 2 + 1, 1 << 42)
    assert taken(L, 4, 2, 64, far // 4, 64, 128, 64, 1 << 42) and not taken(L, 4, 2, 64, far // 4 + 1, 64, 128, 64, 1 << 42)
    assert taken(L, 4, 2, 64, 128, 64, far // 4, 64, 1 << 42) and not taken(L, 4, 2, 64, 128, 64, far // 4 + 1, 64, 1 << 42)
    # heads times stride beyond 64 bits is refused, not wrapped around
    assert not taken(L, 1, 1 << 23, 2, 0, far, 0, 2, 1 << 42) and not taken(L, 1, 1 << 23, 2, 0, 2, 0, far, 1 << 42)


def test_strides_of_an_axis_of_one_do_not_count(L):
    """What a tensor library gives as the stride of an axis of size one is anything."""
    assert taken(L, 1, 4, 64, 256, 64, 9999, 64, 0)                  # in place, one token
    assert taken(L, 4, 1, 64, 64, 64, 64, 7, 0)                      # ... one head
    assert taken(L, 1, 1, 64, 0, 5, 1 << 50, 1 << 60, 0)
    assert taken(L, 1, 4, 64, 1 << 50, 128, 1 << 52, 128, 64)        # slices of one token's heads
    assert taken(L, 4, 1, 64, 128, 1, 128, 2, -64)
    assert not taken(L, 1, 4, 64, 256, 64, 256, 65, 0)
    assert not taken(L, 4, 1, 64, 64, 64, 65, 64, 0)
    assert not taken(L, 1, 4, 64, 1, 128, 2, 128, 63)
    assert not taken(L, 1, 4, 64, -1, 64, 0, 64, 1 << 20) and not taken(L, 4, 1, 64, 64, 0, 64, -1, 1 << 20)
