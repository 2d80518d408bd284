"""What the attention over all visible rows and the norms refuse, with operands that are
apart from each other: what each call is refused for is all that is wrong with it."""
import ctypes as C
import math

import pytest

import dsa_sparse_attention_score_gb300 as dsa
from dsa_sparse_attention_score_gb300 import build as dsa_build

INVALID, UNSUPPORTED, MISALIGNED, SMALL = (dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED,
                                           dsa.DSA_ERR_MISALIGNED, dsa.DSA_ERR_WORKSPACE_TOO_SMALL)
P = C.c_void_p
Q, R, KV, OUT, LSE, WS = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000, 0x6000000   # never dereferenced
GOOD = dict(batch=2, total_q=2, max_q_per_seq=1, max_kv=100, cache_rows=200, cu_q=0x1000, q_pos=0x2000, kv_off=0x3000)


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


def batch(**kw):
    d = dict(GOOD, **kw)
    return dsa.dsa_batch_t(*[d[k] for k in GOOD])


def attn(L, q=Q, r=R, kv=KV, b=None, page=None, H=64, window=None, sinks=0, s0=None, out=OUT, dt=2, lse=LSE, ws=WS, nws=1 << 40):
    a = (P(q), P(r), P(kv), C.byref(b if b is not None else batch()), C.byref(dsa.dsa_paging_t(*page)) if page else None, H)
    z = (0.1, P(out), dt, P(lse), P(ws), nws, None)
    return L.dsa_mla_attn(*a, *z) if window is None else L.dsa_mla_attn_window(*a, window, sinks, P(s0), *z)


# Every call below is refused before the workspace's size is looked at, or for it: with a
# workspace of 0 bytes nothing can be launched, and a call in order answers SMALL.
def refused(L, **kw):
    return attn(L, nws=0, **kw)


@pytest.mark.parametrize("window", [None, 7])
def test_attention(L, window):
    assert refused(L, window=window) == SMALL
    assert refused(L, window=window, r=None, lse=None, dt=0, page=(0x5000, 2, 64)) == SMALL
    for kw in (dict(q=None), dict(kv=None), dict(out=None), dict(dt=1), dict(dt=7), dict(dt=-1), dict(b=batch(batch=0)),
               dict(b=batch(total_q=0)), dict(b=batch(total_q=3)), dict(b=batch(max_q_per_seq=0)), dict(b=batch(cu_q=None)),
               dict(b=batch(q_pos=None)), dict(b=batch(kv_off=None)), dict(b=batch(max_kv=0)), dict(b=batch(cache_rows=0)),
               dict(page=(None, 2, 64)), dict(page=(0x5000, 0, 64)), dict(page=(0x5000, 1, 64)), dict(page=(0x5000, 2, 0))):
        assert refused(L, window=window, **kw) == INVALID, kw
    for kw in (dict(H=0), dict(H=129), dict(b=batch(total_q=1 << 26, max_q_per_seq=1 << 26)),
               dict(b=batch(total_q=1 << 23, max_q_per_seq=1 << 23, max_kv=1 << 30))):
        assert refused(L, window=window, **kw) == UNSUPPORTED, kw
    for kw in (dict(q=Q + 8), dict(r=R + 8), dict(kv=KV + 4), dict(out=OUT + 8), dict(lse=LSE + 2), dict(page=(0x5002, 2, 64))):
        assert refused(L, window=window, **kw) == MISALIGNED, kw
    assert attn(L, window=window, ws=WS + 16) == MISALIGNED and attn(L, window=window, ws=None) == INVALID


def test_window(L):
    for kw in (dict(window=0), dict(window=-3), dict(window=5, sinks=-1)):
        assert refused(L, **kw) == INVALID, kw
    assert refused(L, window=5, sinks=2, s0=0x7002) == MISALIGNED
    assert refused(L, window=2 ** 31 - 1, sinks=2 ** 31 - 1, s0=0x7004) == SMALL


def norm8(L, x=0x1000000, xs=512, r=None, s=0x2000000, w=0x3000000, wt=2, eps=1e-6, codes=0x4000000, scale=0x5000000, group=128,
          dt=2, n=4, dim=512):
    return L.dsa_rms_norm_q8(P(x), xs, P(r), xs, P(s), xs, P(w), wt, eps, P(codes), P(scale), group, dt, n, dim, None)


def test_codes(L):
    for kw in (dict(x=None), dict(codes=None), dict(scale=None), dict(group=0), dict(group=-128), dict(group=100), dict(dim=0),
               dict(dim=-512), dict(n=0), dict(n=-1), dict(wt=1), dict(wt=7), dict(dt=3), dict(dt=-1), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(xs=-4), dict(xs=511)):
        assert norm8(L, **kw) == INVALID, kw
    for kw in (dict(group=256), dict(group=16), dict(dim=520, group=520, xs=520), dict(dim=16400, group=16400, xs=16400)):
        assert norm8(L, **kw) == UNSUPPORTED, kw
    for kw in (dict(x=0x1000001), dict(s=0x2000001), dict(w=0x3000001), dict(w=0x3000002, wt=0), dict(codes=0x4000008),
               dict(scale=0x5000002)):
        assert norm8(L, **kw) == MISALIGNED, kw
