"""What the attention over all visible rows and the norms refuse, before anything
touches a device."""
import ctypes as C
import math

import pytest

import dsa_sparse_attention_score_gb300 as dsa
from dsa_sparse_attention_score_gb300 import build as dsa_build

INVALID, UNSUPPORTED, MISALIGNED, SMALL = (dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED,
                                           dsa.DSA_ERR_MISALIGNED, dsa.DSA_ERR_WORKSPACE_TOO_SMALL)
P = C.c_void_p
X, WS = 0x40000, P(0x10000)                          # never dereferenced: every call fails validation


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


def _batch(**kw):
    d = dict(batch=2, total_q=2, max_q_per_seq=1, max_kv=100, cache_rows=200, cu_q=0x1000, q_pos=0x2000, kv_off=0x3000)
    d.update(kw)
    return dsa.dsa_batch_t(*[d[k] for k in ("batch", "total_q", "max_q_per_seq", "max_kv", "cache_rows", "cu_q", "q_pos",
                                            "kv_off")])


def _attn(L, q=X, r=X, kv=X, batch=None, page=None, H=64, window=None, sinks=0, s0=None, out=X, dt=2, lse=X, ws=WS, nws=1 << 40):
    b = C.byref(batch if batch is not None else _batch())
    pg = C.byref(dsa.dsa_paging_t(*page)) if page else None
    a = (P(q), P(r), P(kv), b, pg, H)
    z = (0.1, P(out), dt, P(lse), ws, nws, None)
    return L.dsa_mla_attn(*a, *z) if window is None else L.dsa_mla_attn_window(*a, window, sinks, P(s0), *z)


@pytest.mark.parametrize("window", [None, 7])
def test_attention_refusals(L, window):
    call = lambda **kw: _attn(L, window=window, **kw)  # noqa: E731
    for kw in (dict(q=None), dict(kv=None), dict(out=None), dict(dt=1), dict(dt=7), dict(ws=P(None)), dict(batch=_batch(batch=0)),
               dict(batch=_batch(total_q=0)), dict(batch=_batch(total_q=3)), dict(batch=_batch(cu_q=None)), dict(batch=_batch(kv_off=None)),
               dict(page=(None, 2, 64)), dict(page=(0x5000, 0, 64)), dict(page=(0x5000, 1, 64)), dict(page=(0x5000, 2, 0)),
               dict(batch=_batch(max_kv=0)), dict(batch=_batch(cache_rows=0))):
        assert call(**kw) == INVALID, kw
    assert L.dsa_mla_attn(P(X), P(X), P(X), None, None, 64, 0.1, P(X), 2, None, WS, 1 << 40, None) == INVALID
    for kw in (dict(H=0), dict(H=129), dict(batch=_batch(total_q=1 << 26, max_q_per_seq=1 << 26)),
               dict(batch=_batch(total_q=1 << 23, max_q_per_seq=1 << 23, max_kv=1 << 30))):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(q=X + 8), dict(r=X + 8), dict(kv=X + 4), dict(out=X + 8), dict(lse=X + 2), dict(ws=P(0x10010)),
               dict(page=(0x5002, 2, 64))):
        assert call(**kw) == MISALIGNED, kw
    assert call(nws=4096) == SMALL


def test_window_refusals(L):
    assert _attn(L, window=0) == INVALID and _attn(L, window=-3) == INVALID and _attn(L, window=5, sinks=-1) == INVALID
    assert _attn(L, window=5, sinks=2, s0=0x6002) == MISALIGNED


def test_attention_workspace(L):
    n = C.c_size_t()
    size = lambda H=64, **kw: (L.dsa_workspace_size(dsa.DSA_OP_MLA_ATTN, C.byref(_batch(**kw)), 1, H, 1, C.byref(n)), n.value)  # noqa: E731
    assert size()[0] == dsa.DSA_OK and size()[1] % 256 == 0
    assert size(H=129)[0] == UNSUPPORTED
    # parts of 152 pieces of 128 rows in float32, and what the plan needs
    parts = 2 * 76 * 128 * (512 + 16 + 2) * 4
    assert parts < size()[1] < parts + (1 << 16)
    assert size(total_q=4096, max_q_per_seq=4096)[1] < parts + (1 << 20)
    assert size(max_kv=1 << 20)[1] == size()[1]          # independent of the context
    assert _attn(L, nws=size()[1] - 1) == SMALL


def _norm(L, x=X, xs=512, r=0x800000, rs=512, s=0x1000000, ss=512, w=0x8000, wt=2, eps=1e-6, out=0x2000000, os=512, dt=2, n=4, dim=512):
    return L.dsa_rms_norm(P(x), xs, P(r), rs, P(s), ss, P(w), wt, eps, P(out), os, dt, n, dim, None)


def _norm8(L, x=X, xs=512, s=0x1000000, w=0x8000, wt=2, eps=1e-6, codes=0x2000000, scale=0x8000, group=128, dt=2, n=4, dim=512):
    return L.dsa_rms_norm_q8(P(x), xs, None, 0, P(s), 512, P(w), wt, eps, P(codes), P(scale), group, dt, n, dim, None)


def test_norm_refusals(L):
    for kw in (dict(x=None), dict(out=None), dict(dt=3), dict(dt=-1), dict(wt=1), dict(wt=5), dict(n=0), dict(dim=0), dict(dim=-8),
               dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(xs=-1), dict(rs=-512), dict(ss=511), dict(os=100),
               dict(xs=1 << 40), dict(os=1 << 41), dict(out=0x1000000), dict(out=X + 2), dict(out=X, os=520), dict(s=0x800000 + 1024),
               dict(out=X + 1024, os=520, xs=520), dict(out=0x1000000 + 100 * 2, os=600, ss=600)):
        assert _norm(L, **kw) == INVALID, kw
    assert _norm(L, dim=16385, xs=20000, rs=20000, ss=20000, os=20000) == UNSUPPORTED
    for kw in (dict(x=X + 1), dict(r=0x800001), dict(s=0x1000001), dict(out=0x2000001), dict(w=0x8001), dict(w=0x8002, wt=0)):
        assert _norm(L, **kw) == MISALIGNED, kw


def test_norm_q8_refusals(L):
    for kw in (dict(x=None), dict(codes=None), dict(scale=None), dict(group=0), dict(group=-128), dict(group=100), dict(dim=0), dict(n=0),
               dict(wt=1), dict(eps=-1.0), dict(xs=-4)):
        assert _norm8(L, **kw) == INVALID, kw
    for kw in (dict(group=256), dict(group=16), dict(dim=520, group=520, xs=520), dict(dim=16400, group=16400, xs=16400)):
        assert _norm8(L, **kw) == UNSUPPORTED, kw
    for kw in (dict(codes=0x2000008), dict(scale=0x8002)):
        assert _norm8(L, **kw) == MISALIGNED, kw


def test_outputs_that_share_memory_are_refused(L):
    # 2 tokens x 64 heads: q_lat and a bf16 out 131,072 bytes, q_rope 16,384, the cache 200 x 1152, lse 512
    far = dict(q=0x100000, r=0x200000, kv=0x300000, out=0x400000, lse=0x500000)
    for kw in (dict(out=0x100000), dict(out=0x100000 + 131072 - 16), dict(out=0x200000 + 16384 - 16), dict(out=0x300000 + 200 * 1152 - 16),
               dict(lse=0x100000), dict(lse=0x300000 + 4), dict(lse=0x400000 + 131072 - 4), dict(out=0x100000 - 131072 + 16)):
        assert _attn(L, **dict(far, **kw)) == INVALID, kw
    for kw in (dict(codes=X), dict(codes=X + 4 * 1024 - 16), dict(codes=0x1000000 - 16), dict(scale=X + 8), dict(scale=0x1000000),
               dict(scale=0x2000000 + 4 * 512 - 4)):
        assert _norm8(L, **kw) == INVALID, kw


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 512, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        dsa.dsa_rms_norm(x, None, None, None, 1e-6, x)
    with pytest.raises(TypeError):
        dsa.dsa_rms_norm_q8(x, None, None, None, 1e-6, torch.zeros(4, 512, dtype=torch.uint8), torch.zeros(4, 4))
    z = torch.zeros(1, dtype=torch.int32)
    b = dsa.Batch(torch.zeros(2, dtype=torch.int32), z, torch.zeros(1, dtype=torch.int64), 1, 1, 4)
    q = torch.zeros(1, 8, 512, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        dsa.dsa_mla_attn(q, None, x, b, 0.1, q, None, x)
