"""The norms' weight may not lie in what they write, which other rows still read it for;
beside column slices of wider rows it may."""
import ctypes as C

import pytest

import dsa_sparse_attention_score_gb300 as dsa
from dsa_sparse_attention_score_gb300 import build as dsa_build

INVALID, UNSUPPORTED = dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED
P = C.c_void_p
X, S, W, OUT, SCALE = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000   # never dereferenced
N, DIM = 4, 512                                      # rows of 1024 bytes in bf16


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


def norm(L, w, wt=2, ss=DIM, os=DIM, n=N, dim=DIM):
    return L.dsa_rms_norm(P(X), DIM, None, 0, P(S), ss, P(w), wt, 1e-6, P(OUT), os, 2, n, dim, None)


def codes(L, w, wt=2, group=128):
    return L.dsa_rms_norm_q8(P(X), DIM, None, 0, P(S), DIM, P(w), wt, 1e-6, P(OUT), P(SCALE), group, 2, N, DIM, None)


@pytest.mark.parametrize("base", [S, OUT])
def test_weight_inside_rows_that_are_written(L, base):
    for w in (base, base + 1024, base + 3 * 1024 + 1022, base - 1022, base + 2):
        assert norm(L, w) == INVALID, hex(w)
    assert norm(L, base - 2044, wt=0) == INVALID     # float32: twice as long
    # slices of rows of 1100 values: column 512 to 1024 is free, 589 on reaches the next row
    for at in (511, 589, 1099):
        w = base + 2 * at
        assert norm(L, w, ss=1100, os=1100) == INVALID, at
        assert norm(L, w + 2 * 1100, ss=1100, os=1100) == INVALID, at
    assert norm(L, base + 2 * 512, wt=0, ss=1100, os=1100) == INVALID
    assert norm(L, base, n=1) == INVALID


def test_weight_inside_codes_and_scales(L):
    for w in (S, S + 4 * 1024 - 2, OUT, OUT + N * DIM - 2, OUT - 1022, SCALE, SCALE + 4 * 4 * N - 4, SCALE - 1020):
        assert codes(L, w) == INVALID, hex(w)
        assert codes(L, w // 4 * 4, wt=0) == INVALID, hex(w)


@pytest.mark.gpu
def test_weight_beside_the_rows_that_are_written():
    import torch
    big = torch.randn(40, 1100, device="cuda").bfloat16()
    big[7, 530:1042] = 1 + 0.1 * torch.randn(512, device="cuda").bfloat16()
    w, before = big[7, 530:1042], big.clone()
    dsa.dsa_rms_norm(big[:, :512], None, None, w, 1e-6, big[:, :512])
    x = before[:, :512].double()
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6) * before[7, 530:1042].double()
    assert torch.equal(big[:, 512:], before[:, 512:])
    assert ((big[:, :512].double() - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -17)).all()
