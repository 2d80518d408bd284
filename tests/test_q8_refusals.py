"""Rotary positions and the 8-bit cache: the host's frequencies and what the
calls refuse, before anything touches a device."""
import ctypes as C
import math

import pytest

import dsa_sparse_attention_score_gb300 as dsa
from dsa_sparse_attention_score_gb300 import build as dsa_build

INVALID, UNSUPPORTED, MISALIGNED, SMALL = (dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED,
                                           dsa.DSA_ERR_MISALIGNED, dsa.DSA_ERR_WORKSPACE_TOO_SMALL)
P = C.c_void_p
X, WS, NWS = P(0x40000), P(0x10000), 1 << 30        # never dereferenced: every call fails validation


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


def _batch(**kw):
    d = dict(batch=2, total_q=2, max_q_per_seq=1, max_kv=100, cache_rows=200, cu_q=0x1000, q_pos=0x2000, kv_off=0x3000)
    d.update(kw)
    return dsa.dsa_batch_t(*[d[k] for k in ("batch", "total_q", "max_q_per_seq", "max_kv", "cache_rows", "cu_q", "q_pos",
                                            "kv_off")])


# ------------------------------------------------------------- frequencies

def test_plain_and_linear_frequencies(L):
    f, s = dsa.dsa_rope_frequencies(64, 10000.0)
    assert s == 1.0 and len(f) == 32
    for j, v in enumerate(f):
        assert v == pytest.approx(10000.0 ** (-2 * j / 64), rel=1e-15)
    g, s = dsa.dsa_rope_frequencies(64, 10000.0, "linear", 4.0)
    assert s == 1.0 and all(b == pytest.approx(a / 4, rel=1e-15) for a, b in zip(f, g))


def test_ntk_keeps_the_fastest_pair_and_divides_the_slowest(L):
    f, _ = dsa.dsa_rope_frequencies(128, 10000.0)
    g, s = dsa.dsa_rope_frequencies(128, 10000.0, "ntk", 8.0)
    assert s == 1.0 and g[0] == f[0]
    # base factor^(d/(d-2)): the slowest pair, exponent -(d-2)/d, is divided by factor
    assert g[-1] == pytest.approx(f[-1] / 8.0, rel=1e-12)


def test_yarn_blends_between_the_two(L):
    f, _ = dsa.dsa_rope_frequencies(64, 10000.0)
    g, s = dsa.dsa_rope_frequencies(64, 10000.0, "yarn", 40.0, 4096, 32.0, 1.0)
    assert s == pytest.approx(0.1 * math.log(40.0) + 1.0, rel=1e-6)
    at = lambda beta: 64 * math.log(4096 / (beta * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    low, high = math.floor(at(32.0)), math.ceil(at(1.0))
    for j in range(32):
        r = min(1.0, max(0.0, (j - low) / (high - low)))
        assert g[j] == pytest.approx(f[j] * (1 - r) + f[j] / 40.0 * r, rel=1e-14), j
    assert g[0] == f[0] and g[-1] == pytest.approx(f[-1] / 40.0, rel=1e-14)
    assert dsa.dsa_rope_frequencies(64, 10000.0, "yarn", 1.0)[0] == pytest.approx(f, rel=1e-15)


def test_frequency_refusals(L):
    f, s = (C.c_double * 256)(), C.c_float()
    call = lambda rot=64, base=1e4, sc=0, factor=2.0, ctx=4096, bf=32.0, bs=1.0, out=f, sp=None: L.dsa_rope_frequencies(  # noqa: E731
        rot, base, sc, factor, ctx, bf, bs, out, C.byref(s) if sp is None else sp)
    assert call() == dsa.DSA_OK
    for kw in (dict(rot=0), dict(rot=63), dict(rot=-2), dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(sc=4),
               dict(sc=-1), dict(sc=1, factor=0.5), dict(sc=3, factor=math.nan), dict(sc=2, rot=2), dict(sc=3, ctx=0),
               dict(sc=3, bf=1.0, bs=1.0), dict(sc=3, bs=0.0), dict(out=None), dict(sp=P(None))):
        assert call(**kw) == INVALID, kw
    assert call(rot=514) == UNSUPPORTED
    assert call(sc=0, factor=0.0) == dsa.DSA_OK            # no scaling: the factor is not read
    with pytest.raises(ValueError):
        dsa.dsa_rope_frequencies(64, 1e4, "dynamic")


# -------------------------------------------------------------- rope calls

def _rope_call(L, x=0x40000, xt=512, xh=64, y=0x900000, yt=512, yh=64, dt=2, T=4, H=8, D=64, off=0, pos=X, f=0x8000, rot=64,
               rope=True):
    r = dsa.dsa_rope_t(f, rot, 1, 1.0)
    return L.dsa_rope(P(x), xt, xh, P(y), yt, yh, dt, T, H, D, off, pos, C.byref(r) if rope else None, 0, None)


def test_rope_refusals(L):
    for kw in (dict(x=0), dict(y=0), dict(pos=None), dict(rope=False), dict(dt=3), dict(dt=-1), dict(T=0), dict(H=0), dict(D=1),
               dict(off=-1), dict(off=2), dict(rot=63), dict(rot=0), dict(rot=66), dict(f=0), dict(xt=-1), dict(xh=-1),
               dict(yt=-1), dict(yh=-8), dict(yh=63), dict(yt=0), dict(yt=500), dict(yh=0), dict(xt=1 << 62)):
        assert _rope_call(L, **kw) == INVALID, kw
    assert _rope_call(L, D=1024, rot=514) == UNSUPPORTED
    assert _rope_call(L, H=1 << 20, D=64, yt=1 << 26, xt=1 << 26) == UNSUPPORTED
    for kw in (dict(x=0x40001), dict(y=0x900001), dict(dt=0, x=0x40002), dict(pos=P(0x40002)), dict(f=0x8004)):
        assert _rope_call(L, **kw) == MISALIGNED, kw


def test_rope_refuses_memory_that_overlaps(L):
    n = 2 * (4 * 512)                                      # bytes of x
    assert _rope_call(L, y=0x40000, yt=1024) == INVALID    # same start, other strides
    assert _rope_call(L, y=0x40000 + n - 2) == INVALID     # the last value
    assert _rope_call(L, y=0x40000 + 2) == INVALID         # one value on
    # slices of one buffer's heads that overlap: 64 values apart by 32
    assert _rope_call(L, xt=8 * 192, xh=192, y=0x40000 + 64, yt=8 * 192, yh=192) == INVALID
    # a slice that would reach into the next head
    assert _rope_call(L, xt=8 * 100, xh=100, y=0x40000 + 2 * 64, yt=8 * 100, yh=100) == INVALID


# ------------------------------------------------------------- cache calls

def test_append_refusals(L):
    b, r = _batch(), dsa.dsa_rope_t(0x8000, 64, 1, 1.0)

    def call(c=X, cs=576, rn=X, rs=576, dt=2, batch=b, pg=None, rope=C.byref(r), codes=X, scale=X, ws=WS, n=NWS):
        q8 = L.dsa_kv_append_q8(c, cs, rn, rs, dt, C.byref(batch) if batch else None, pg, rope, codes, scale, ws, n, None)
        b16 = L.dsa_kv_append(c, cs, rn, rs, dt, C.byref(batch) if batch else None, pg, rope, codes, ws, n, None)
        return q8, b16

    for kw in (dict(c=None), dict(codes=None), dict(dt=5), dict(batch=None), dict(cs=-1), dict(rs=-1), dict(rn=None),
               dict(batch=_batch(total_q=3)), dict(batch=_batch(kv_off=0)), dict(batch=_batch(max_kv=0)), dict(ws=None)):
        assert call(**kw) == (INVALID, INVALID), kw
    assert call(scale=None)[0] == INVALID
    for rot in (32, 128):
        assert call(rope=C.byref(dsa.dsa_rope_t(0x8000, rot, 1, 1.0))) == (UNSUPPORTED, UNSUPPORTED)
    assert call(rope=C.byref(dsa.dsa_rope_t(0, 64, 1, 1.0))) == (INVALID, INVALID)
    for kw in (dict(c=P(0x40001)), dict(rn=P(0x40001)), dict(codes=P(0x40008)), dict(dt=0, c=P(0x40002)), dict(ws=P(0x10010))):
        assert call(**kw) == (MISALIGNED, MISALIGNED), kw
    assert call(scale=P(0x40002))[0] == MISALIGNED
    assert call(n=16) == (SMALL, SMALL)
    for pg, want in ((dsa.dsa_paging_t(None, 2, 64), INVALID), (dsa.dsa_paging_t(0x40000, 1, 64), INVALID),
                     (dsa.dsa_paging_t(0x40000, 2, 0), INVALID), (dsa.dsa_paging_t(0x40000, 0, 64), INVALID),
                     (dsa.dsa_paging_t(0x40002, 2, 64), MISALIGNED)):
        assert call(pg=C.byref(pg)) == (want, want)


def test_read_refusals(L):
    b = _batch()

    def call(codes=X, scale=X, tail=1, batch=b, out=X, dt=2, stride=576, ws=WS, n=NWS):
        return L.dsa_kv_read_q8(codes, scale, tail, C.byref(batch), None, out, dt, stride, ws, n, None)

    for kw in (dict(codes=None), dict(scale=None), dict(out=None), dict(dt=1), dict(stride=575), dict(stride=-576),
               dict(tail=0, stride=511), dict(batch=_batch(cache_rows=1 << 31)), dict(ws=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(codes=P(0x40004)), dict(scale=P(0x40002)), dict(out=P(0x40001)), dict(dt=0, out=P(0x40002))):
        assert call(**kw) == MISALIGNED, kw
    assert call(n=255) == SMALL


def test_attention_refusals(L):
    b = _batch()

    def call(q=X, qr=X, codes=X, scale=X, batch=b, pg=None, idx=X, k=16, H=8, out=X, dt=2, lse=None, ws=WS, n=NWS):
        return L.dsa_sparse_mla_attn_q8(q, qr, codes, scale, C.byref(batch), pg, idx, k, H, 0.1, out, dt, lse, ws, n, None)

    for kw in (dict(q=None), dict(codes=None), dict(scale=None), dict(idx=None), dict(out=None), dict(dt=1), dict(ws=None),
               dict(batch=_batch(q_pos=0)), dict(pg=C.byref(dsa.dsa_paging_t(0x40000, 1, 64)))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(k=0), dict(k=65537), dict(H=0), dict(H=129)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(q=P(0x40008)), dict(qr=P(0x40008)), dict(codes=P(0x40008)), dict(out=P(0x40004)), dict(idx=P(0x40002)),
               dict(lse=P(0x40002)), dict(ws=P(0x10080))):
        assert call(**kw) == MISALIGNED, kw
    n = C.c_size_t()
    assert L.dsa_workspace_size(dsa.DSA_OP_SPARSE_ATTN, C.byref(b), 1, 8, 16, C.byref(n)) == dsa.DSA_OK
    assert call(n=n.value - 1) == SMALL


def test_binding_checks_shapes_before_the_call():
    import torch

    class Fake:                                # stands in for a CUDA tensor; no GPU needed
        device = "cuda:0"

        def __init__(self, dtype, *shape):
            self.dtype, self.shape = dtype, torch.Size(shape)

        def get_device(self):
            return 0

        def is_contiguous(self):
            return True

        def numel(self):
            return self.shape.numel()

        def data_ptr(self):
            return 0x1000

        def stride(self, i=None):
            st = [self.shape[j + 1:].numel() for j in range(len(self.shape))]
            return st if i is None else st[i]

    b = dsa.Batch(Fake(torch.int32, 4), Fake(torch.int32, 3), Fake(torch.int64, 3), 1, 100, 200)
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    codes, scale = Fake(u8, 200, 640), Fake(f32, 200)
    with pytest.raises(TypeError, match="codes"):          # a cache of rows without a tail, and a tail
        dsa.dsa_kv_append_q8(Fake(bf, 3, 512), Fake(bf, 3, 64), b, None, Fake(u8, 200, 512), scale, None)
    with pytest.raises(TypeError, match="scale"):
        dsa.dsa_kv_append_q8(Fake(bf, 3, 512), Fake(bf, 3, 64), b, None, codes, Fake(f32, 199), None)
    with pytest.raises(TypeError, match="names 200"):
        dsa.dsa_kv_append_q8(Fake(bf, 3, 512), Fake(bf, 3, 64), b, None, Fake(u8, 199, 640), Fake(f32, 199), None)
    with pytest.raises(TypeError, match="c_new"):
        dsa.dsa_kv_append_q8(Fake(bf, 4, 512), Fake(bf, 3, 64), b, None, codes, scale, None)
    with pytest.raises(TypeError, match="r_new"):
        dsa.dsa_kv_append_q8(Fake(bf, 3, 512), Fake(f32, 3, 64), b, None, codes, scale, None)
    with pytest.raises(TypeError, match="kv_cache"):
        dsa.dsa_kv_append(Fake(bf, 3, 512), Fake(bf, 3, 64), b, None, Fake(bf, 200, 512), None)
    with pytest.raises(TypeError, match="out"):
        dsa.dsa_kv_read_q8(codes, scale, b, Fake(bf, 3, 512), None)
    with pytest.raises(TypeError, match="out"):
        dsa.dsa_kv_read_q8(codes, scale, b, Fake(torch.float16, 3, 576), None)
    with pytest.raises(TypeError, match="q_lat"):
        dsa.dsa_sparse_mla_attn_q8(Fake(bf, 2, 8, 512), None, codes, scale, b, Fake(torch.int32, 3, 4), 1.0,
                                   Fake(bf, 3, 8, 512), None, None)
    with pytest.raises(TypeError, match="codes"):
        dsa.dsa_sparse_mla_attn_q8(Fake(bf, 3, 8, 512), None, codes, scale, b, Fake(torch.int32, 3, 4), 1.0,
                                   Fake(bf, 3, 8, 512), None, None)
    with pytest.raises(TypeError, match="kv_off"):
        wrong = dsa.Batch(b.cu_q, b.q_pos, Fake(torch.int32, 3), 1, 100, 200)
        dsa.dsa_kv_read_q8(codes, scale, wrong, Fake(bf, 3, 576), None)
    with pytest.raises(TypeError, match="block_table"):
        dsa.dsa_kv_read_q8(codes, scale, b, Fake(bf, 3, 576), None, Fake(torch.int32, 2, 4), 64)
    with pytest.raises(TypeError, match="x, out"):
        dsa.dsa_rope(Fake(bf, 3, 8, 64), Fake(torch.int32, 3), None, Fake(f32, 3, 8, 64))
    with pytest.raises(TypeError, match="pos"):
        dsa.dsa_rope(Fake(bf, 3, 8, 64), Fake(torch.int32, 4), None, Fake(bf, 3, 8, 64))
