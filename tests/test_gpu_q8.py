"""Rotary positions, the 8-bit latent cache and the attention over it on the
GPU against float64 (tests/_q8_ref.py, which derives the bounds)."""
import numpy as np
import pytest

import _q8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    from dsa_sparse_attention_score_gb300 import build
    build.build()
    import dsa_sparse_attention_score_gb300 as m
    return m


@pytest.fixture(scope="module")
def torch():
    import torch as t
    return t


def dt_of(torch, name):
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(torch, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------- rope

ROPE = [
    # T, heads, dim, rot_off, rot_dim, dtype, interleaved, inverse, scaling
    (1, 1, 64, 0, 64, "bf16", True, False, "none"),
    (5, 64, 64, 0, 64, "bf16", True, False, "yarn"),
    (33, 8, 128, 0, 64, "f16", False, False, "linear"),
    (33, 8, 128, 64, 64, "f16", True, True, "none"),
    (7, 3, 192, 128, 64, "f32", False, True, "ntk"),
    (3, 5, 70, 3, 64, "bf16", True, False, "none"),       # no 16-byte units
    (3, 5, 71, 4, 66, "f32", False, False, "none"),
    (2, 2, 513, 1, 512, "f16", False, False, "none"),
    (2, 130, 2, 0, 2, "bf16", True, False, "none"),
    (2, 130, 10, 2, 2, "f32", False, False, "none"),
    (700, 128, 96, 32, 32, "bf16", False, False, "yarn"),
    (2, 200, 256, 0, 256, "f32", True, False, "none"),    # several CTAs per token
]


def rope_check(torch, x, out, pos, rope, rot_off, inverse, dtype):
    xs, y = f64(x), f64(out)
    n = rope.rot_dim
    ref, size = R.rotate(xs[..., rot_off:rot_off + n], pos, f64(rope.inv_freq), rope.scale, rope.interleaved, inverse)
    got = y[..., rot_off:rot_off + n]
    assert np.all(np.abs(got - ref) <= R.HALF_STEP[dtype] * np.abs(ref) + 2.0 ** -20 * size + 2.0 ** -25 * (dtype == "f16"))
    rest = np.ones(xs.shape[-1], bool)
    rest[rot_off:rot_off + n] = False
    assert np.array_equal(y[..., rest], xs[..., rest])


@pytest.mark.parametrize("T,heads,dim,off,rot,dtype,inter,inverse,scaling", ROPE)
def test_rope(dsa, torch, T, heads, dim, off, rot, dtype, inter, inverse, scaling):
    g = gen(torch, T * heads + dim)
    x = torch.randn(T, heads, dim, generator=g, device="cuda").to(dt_of(torch, dtype))
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    rope = dsa.Rope.make(rot, 1e4, inter, scaling, 8.0, 4096)
    out = torch.full_like(x, float("nan"))
    dsa.dsa_rope(x, pos, rope, out, off, inverse)
    rope_check(torch, x, out, pos.cpu().numpy(), rope, off, inverse, dtype)
    # in place: the same bits, nothing else touched
    y = x.clone()
    dsa.dsa_rope(y, pos, rope, y, off, inverse)
    assert torch.equal(y, out)


def test_rope_strides_and_slices(dsa, torch):
    g = gen(torch, 7)
    rope = dsa.Rope.make(64, 1e4, True)
    pos = torch.tensor([0, 3, 100, -5, 77], dtype=torch.int32, device="cuda")
    big = torch.randn(5, 12, 200, generator=g, device="cuda").to(torch.bfloat16)
    keep = big.clone()
    for x in (big[:, :, 128:192], big[:, 2:9, 8:72], big[:, :, 3:67], big.transpose(0, 1)[:5, :5, :64]):
        T = x.shape[0]
        out = torch.empty(x.shape, dtype=x.dtype, device="cuda")
        dsa.dsa_rope(x, pos[:T].contiguous(), rope, out)
        rope_check(torch, x, out, pos[:T].cpu().numpy(), rope, 0, False, "bf16")
    assert torch.equal(big, keep)
    # one slice of each head into another: the rest of the buffer stays
    dsa.dsa_rope(big[:, :, 0:64], pos, rope, big[:, :, 64:128])
    rope_check(torch, keep[:, :, 0:64], big[:, :, 64:128], pos.cpu().numpy(), rope, 0, False, "bf16")
    assert torch.equal(big[:, :, :64], keep[:, :, :64]) and torch.equal(big[:, :, 128:], keep[:, :, 128:])
    # a broadcast input: one row for every head and token
    one = torch.randn(1, 1, 64, generator=g, device="cuda").expand(5, 12, 64)
    out = torch.empty(5, 12, 64, device="cuda")
    dsa.dsa_rope(one, pos, rope, out)
    rope_check(torch, one, out, pos.cpu().numpy(), rope, 0, False, "f32")
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rope(out, pos, rope, out[:1, :1].expand(5, 12, 64))


@pytest.mark.parametrize("inter", [True, False])
def test_rope_gradient(dsa, torch, inter):
    """<dy, dsa_rope(x)> as a function of x has the gradient that the inverse
    call gives for dy: against the formula's (the test above) and against
    differences in the output of the forward call itself.  The map is linear,
    so the difference over a step of x is exact up to the call's rounding:
    |<dy, y(x + h e) - y(x)> / h - g| <= 2 * 2^-19 sum |dy| (|a| + |b|) / h."""
    g = gen(torch, 9)
    T, H, D, off, rot = 3, 2, 24, 4, 16
    rope = dsa.Rope.make(rot, 100.0, inter, "yarn", 4.0, 64)
    pos = torch.tensor([1, 50, 1000], dtype=torch.int32, device="cuda")
    x, dy = (torch.randn(T, H, D, generator=g, device="cuda") for _ in range(2))
    grad = torch.empty_like(dy)
    dsa.dsa_rope(dy, pos, rope, grad, off, inverse=True)
    y0 = torch.empty_like(x)
    dsa.dsa_rope(x, pos, rope, y0, off)
    h = 1.0
    for d in range(D):
        xp = x.clone()
        xp[:, :, d] += h
        step = (xp - x)[:, :, d].double()
        y1 = torch.empty_like(x)
        dsa.dsa_rope(xp, pos, rope, y1, off)
        diff = ((y1.double() - y0.double()) * dy.double()).sum(2) / step
        size = 2 * 2.0 ** -19 * rope.scale * (dy.double().abs() * 2 * (x.double().abs().amax(2, keepdim=True) + 1)).sum(2)
        assert torch.all((diff - grad[:, :, d].double()).abs() <= size + 2.0 ** -19 * rope.scale * 2 * dy.double().abs().amax(2))


# ------------------------------------------------------------------ cache

class Seqs:
    """Sequences of given lengths with per[b] new tokens at their ends."""

    def __init__(self, dsa, torch, lens, per, page=0, gap=3, seed=0):
        self.lens, self.per, self.page = lens, per, page
        B = len(lens)
        cu = np.concatenate([[0], np.cumsum(per)])
        pos = np.concatenate([np.arange(n - p, n) for n, p in zip(lens, per)]).astype(np.int32)
        rng = np.random.default_rng(seed)
        if page:
            nb = [-(-n // page) for n in lens]
            perm = rng.permutation(sum(nb) + 2)
            self.table = np.full((B, max(nb)), -1, np.int32)
            at = 0
            for b, n in enumerate(nb):
                self.table[b, :n] = perm[at:at + n]
                at += n
            self.rows, off = (sum(nb) + 2) * page, [0] * B
        else:
            self.table = None
            ends = np.cumsum([n + gap for n in lens])
            off = [0] + [int(e) for e in ends[:-1]]
            self.rows = int(ends[-1])
        self.off, self.pos, self.seq = off, pos, np.repeat(np.arange(B), per)
        self.batch = dsa.Batch.from_host(cu, pos, off, self.rows, max_kv=max(lens))
        self.block = torch.from_numpy(self.table).cuda() if page else None
        self.ws = dsa.workspace(dsa.DSA_OP_K_APPEND, self.batch)

    def row(self, b, p):
        p = np.asarray(p)
        return self.off[b] + p if not self.page else self.table[b, p // self.page].astype(np.int64) * self.page + p % self.page

    def token_rows(self):
        return np.array([int(self.row(b, p)) for b, p in zip(self.seq, self.pos)])

    @property
    def paging(self):
        return (self.block, self.page) if self.page else (None, 0)


def special_rows(x):
    """Rows where a scale can go wrong: zeros, the largest on and beside the
    border 448 * 2^n, far ranges, values under the smallest code."""
    n = x.shape[0]
    x = x.copy()
    put = [0.0, 448.0, 449.0, 447.0, 2.0 ** 60, 2.0 ** -45, 1.75 * 2.0 ** -31, 3e38, 2.0 ** -100]
    for i, top in enumerate(put):
        if i + 1 < n:
            r = x[i + 1]
            m = np.abs(r).max()
            x[i + 1] = r / m * top
            if top:
                x[i + 1, np.argmax(np.abs(r))] = top
    return x


APPEND = [
    # lens, per, page, dtype, tail, interleaved, rotate
    ([40], [1], 0, "bf16", True, True, True),
    ([40, 70, 33], [13, 1, 20], 0, "bf16", True, False, True),
    ([40, 70, 33], [13, 1, 20], 16, "f32", True, True, True),
    ([300, 129], [260, 100], 64, "f16", True, True, False),
    ([300, 129], [260, 100], 1, "f32", False, True, False),
    ([25] * 40, [1] * 40, 7, "bf16", False, True, False),
    ([5000], [5000], 0, "f32", True, False, True),
]


@pytest.mark.parametrize("lens,per,page,dtype,tail,inter,rotate", APPEND)
def test_append_and_read(dsa, torch, lens, per, page, dtype, tail, inter, rotate):
    s = Seqs(dsa, torch, lens, per, page, seed=len(lens))
    T, dt = s.batch.T, dt_of(torch, dtype)
    wide = 576 if tail else 512
    x = np.random.default_rng(1).standard_normal((T, wide))
    x = special_rows(x) if dtype != "f16" else x
    x = torch.from_numpy(x).to(dt).cuda()
    store = torch.full((T, wide + 5), float("nan"), dtype=dt, device="cuda")     # odd row stride: no vector loads
    store[:, :wide] = x
    rope = dsa.Rope.make(64, 1e4, inter, "yarn", 4.0, 32) if rotate else None
    codes0 = torch.randint(0, 256, (s.rows, 640 if tail else 512), dtype=torch.uint8, device="cuda")
    scale0 = torch.rand(s.rows, device="cuda")
    got = []
    for src in (x, store):
        codes, scale = codes0.clone(), scale0.clone()
        dsa.dsa_kv_append_q8(src[:, :512], src[:, 512:wide] if tail else None, s.batch, rope, codes, scale, s.ws, *s.paging)
        assert dsa.dsa_read_device_status(s.ws) == 0
        got.append((codes, scale))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    codes, scale = got[0]
    at = s.token_rows()
    others = np.setdiff1d(np.arange(s.rows), at)
    assert torch.equal(codes[others], codes0[others]) and torch.equal(scale[others], scale0[others])
    lat, r = f64(x)[:, :512], f64(x)[:, 512:] if tail else None
    slack = np.zeros_like(r) if tail else None
    if rotate:
        r, size = R.rotate(r, s.pos, f64(rope.inv_freq), rope.scale, inter)
        slack = 2.0 ** -20 * size
    ref, ref_s = R.quantise(lat, r)
    c, sc = codes[at].cpu().numpy(), f64(scale[at])
    if not rotate:
        assert np.array_equal(sc, ref_s)
        assert np.array_equal(c, R.encode(ref))
    else:
        # a scale may fall on the other side of its border only where the
        # rotated value is within the rotation's error of it
        top = np.maximum(np.abs(lat).max(1), np.abs(r).max(1))
        E, near = R.exponent(top), slack.max(1)
        lo, hi = R.exponent(top - near), R.exponent(top + near)
        got_E = np.log2(sc)
        assert np.all((got_E >= lo) & (got_E <= hi))
        assert (lo == hi).mean() > 0.9
        same = got_E == E
        assert np.array_equal(c[same, :512], R.encode(ref[same, :512]))
        v = R.e4m3_decode(c)[:, 512:] * sc[:, None]
        err = np.abs(v[:, :64] + v[:, 64:] - r)
        clipped = np.abs(r) > 448 * 2.0 ** 119
        assert np.all((err <= 2.0 ** -8 * np.abs(r) + 2.0 ** -10 * sc[:, None] + 2 * slack) | clipped)
    # reading back: code * scale, the tail's sum rounded once
    vlat, vtail = R.decode_rows(c, sc)
    want = np.concatenate([vlat, vtail], 1) if tail else vlat
    for odt, name in ((torch.bfloat16, "bf16"), (torch.float32, "f32")):
        for pad in (0, 3, 8):
            buf = torch.full((T, wide + pad), -7.0, dtype=odt, device="cuda")
            dsa.dsa_kv_read_q8(codes, scale, s.batch, buf[:, :wide], s.ws, *s.paging)
            g = f64(buf)
            assert np.array_equal(g[:, :512], want[:, :512])
            assert np.all(np.abs(g[:, 512:wide] - want[:, 512:]) <= R.HALF_STEP[name] * np.abs(want[:, 512:]))
            assert np.all(g[:, wide:] == -7.0)
    assert dsa.dsa_read_device_status(s.ws) == 0
    # the bf16 cache
    kv0 = torch.randn(s.rows, wide, device="cuda").to(torch.bfloat16)
    kv = kv0.clone()
    dsa.dsa_kv_append(x[:, :512], x[:, 512:] if tail else None, s.batch, rope, kv, s.ws, *s.paging)
    assert torch.equal(kv[others], kv0[others])
    assert torch.equal(kv[at, :512], x[:, :512].to(torch.bfloat16))
    if tail:
        g = f64(kv[at, 512:])
        ok = np.abs(r) < 3.3e38
        assert np.all((np.abs(g - r) <= 2.0 ** -8 * np.abs(r) + slack)[ok])


def test_append_rows_that_are_not_finite(dsa, torch):
    s = Seqs(dsa, torch, [9], [9])
    x = torch.randn(9, 576, device="cuda")
    for i, (col, v) in enumerate([(0, np.nan), (511, np.inf), (512, -np.inf), (575, np.nan)]):
        x[2 * i, col] = float(v)
    codes, scale = dsa.q8_cache(s.rows)
    rope = dsa.Rope.make(64)
    dsa.dsa_kv_append_q8(x[:, :512], x[:, 512:], s.batch, rope, codes, scale, s.ws)
    out = torch.empty(9, 576, device="cuda")
    dsa.dsa_kv_read_q8(codes, scale, s.batch, out, s.ws)
    bad = torch.tensor([0, 2, 4, 6], device="cuda")
    good = torch.tensor([1, 3, 5, 7, 8], device="cuda")
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[good]).all()
    assert torch.isnan(scale[bad]).all() and (codes[bad] == 0).all()


def test_positions_out_of_bounds_are_flagged_and_skipped(dsa, torch):
    """Negative and too large positions, an unmapped block, a row past the cache."""
    for page in (0, 16):
        s = Seqs(dsa, torch, [40, 40], [3, 3], page)
        b = s.batch
        b.q_pos = torch.tensor([5, -1, 40, 7, 2 ** 31 - 1, 39], dtype=torch.int32, device="cuda")
        if page:
            s.block[1, 2] = -1                              # position 39 of sequence 1
        else:
            b.kv_off[1] = s.rows - 39                       # ... or past the last row
        x = torch.randn(6, 576, device="cuda")
        codes0 = torch.randint(0, 127, (s.rows, 640), dtype=torch.uint8, device="cuda")
        codes, scale = codes0.clone(), torch.ones(s.rows, device="cuda")
        dsa.dsa_kv_append_q8(x[:, :512], x[:, 512:], b, None, codes, scale, s.ws, *s.paging)
        assert dsa.dsa_read_device_status(s.ws) == dsa.DSA_DEV_BAD_POSITION
        off = [0, s.rows - 39] if not page else None
        at = [int(s.row(0, 5)), int(s.row(1, 7)) if page else off[1] + 7]
        changed = (codes != codes0).any(1).nonzero()[:, 0].tolist()
        assert sorted(changed) == sorted(at)
        out = torch.full((6, 576), float("nan"), device="cuda")
        dsa.dsa_kv_read_q8(codes, scale, b, out, s.ws, *s.paging)
        assert dsa.dsa_read_device_status(s.ws) == dsa.DSA_DEV_BAD_POSITION
        zero = (out == 0).all(1)
        assert zero.tolist() == [False, True, True, False, True, True]
        idx = torch.zeros(6, 4, dtype=torch.int32, device="cuda")
        q = torch.randn(6, 3, 512, device="cuda").to(torch.bfloat16)
        ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, b, H=3, k=4)
        o, lse = torch.full((6, 3, 512), float("nan"), device="cuda"), torch.zeros(6, 3, device="cuda")
        dsa.dsa_sparse_mla_attn_q8(q, q[:, :, :64].contiguous(), codes, scale, b, idx, 0.1, o, lse, ws, *s.paging)
        assert dsa.dsa_read_device_status(ws) & dsa.DSA_DEV_BAD_POSITION
        for t, bad in enumerate([False, True, True, False, True, True]):
            assert bool((o[t] == 0).all()) == bad and bool(torch.isneginf(lse[t]).all()) == bad


def test_rows_beyond_32_bit_offsets(dsa, torch):
    """A cache of more than 2^31 bytes of codes: the last rows."""
    rows = (1 << 31) // 640 + 5000
    codes, scale = dsa.q8_cache(rows)
    T = 40
    b = dsa.Batch.from_host([0, T], range(T), [rows - T], rows)
    ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, b, H=2, k=T)
    x = torch.randn(T, 576, device="cuda")
    dsa.dsa_kv_append_q8(x[:, :512], x[:, 512:], b, None, codes, scale, ws)
    out = torch.empty(T, 576, device="cuda")
    dsa.dsa_kv_read_q8(codes, scale, b, out, ws)
    assert torch.all((out - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10)
    idx = torch.arange(T, dtype=torch.int32, device="cuda").repeat(T, 1)
    idx = torch.where(idx <= torch.arange(T, device="cuda")[:, None], idx, -1).contiguous()
    q = torch.randn(T, 2, 576, device="cuda").to(torch.bfloat16)
    o = torch.empty(T, 2, 512, device="cuda")
    dsa.dsa_sparse_mla_attn_q8(q[:, :, :512].contiguous(), q[:, :, 512:].contiguous(), codes, scale, b, idx, 0.05, o, None, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    c, sc = codes[-T:].cpu().numpy(), f64(scale[-T:])
    for t in (0, 17, T - 1):
        ref, _, tol, _ = R.attention(f64(q[t, :, :512]), f64(q[t, :, 512:]), c, sc, np.arange(t + 1), 0.05)
        assert np.all(np.abs(f64(o[t]) - ref) <= tol)


# -------------------------------------------------------------- attention

def fill_cache(dsa, torch, s, tail, spread=0.5, seed=3):
    g = gen(torch, seed)
    b = dsa.Batch.from_host([0, s.rows], range(s.rows), [0], s.rows)
    x = torch.randn(s.rows, 576 if tail else 512, generator=g, device="cuda")
    x *= torch.exp2(spread * torch.randn(s.rows, 1, generator=g, device="cuda"))
    codes, scale = dsa.q8_cache(s.rows, tail)
    dsa.dsa_kv_append_q8(x[:, :512], x[:, 512:] if tail else None, b, None, codes, scale, s.ws)
    return codes, scale


def selections(s, k, seed=5, twice=False):
    rng = np.random.default_rng(seed)
    idx = np.full((len(s.pos), k), -1, np.int32)
    for t, p in enumerate(s.pos):
        n = min(k, int(p) + 1)
        idx[t, :n] = np.sort(rng.choice(int(p) + 1, n, replace=False))
        if twice and n > 2:
            idx[t, 1] = idx[t, 0]
    return idx


def attend(dsa, torch, s, H, k, idx, tail=True, spread=0.5, size=1.0, out_dt="f32", check=None, sm=1 / 13.86, with_lse=True):
    codes, scale = fill_cache(dsa, torch, s, tail, spread)
    g = gen(torch, 11)
    T = s.batch.T
    q = (size * torch.randn(T, H, 512, generator=g, device="cuda")).to(torch.bfloat16)
    qr = (size * torch.randn(T, H, 64, generator=g, device="cuda")).to(torch.bfloat16) if tail else None
    ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=H, k=k)
    out = torch.full((T, H, 512), float("nan"), dtype=dt_of(torch, out_dt), device="cuda")
    lse = torch.full((T, H), float("nan"), device="cuda") if with_lse else None
    dsa.dsa_sparse_mla_attn_q8(q, qr, codes, scale, s.batch, torch.from_numpy(idx).cuda(), sm, out, lse, ws, *s.paging)
    assert dsa.dsa_read_device_status(ws) == 0
    go, c, sc = f64(out), codes.cpu().numpy(), f64(scale)
    gl = f64(lse) if with_lse else None
    qa, qb = f64(q), f64(qr) if tail else None
    for t in range(T) if check is None else check:
        sel = idx[t][idx[t] >= 0]
        rows = np.asarray(s.row(int(s.seq[t]), sel))
        ref, rl, tol, tl = R.attention(qa[t], qb[t] if tail else None, c, sc, rows, sm)
        half = R.HALF_STEP[out_dt] * np.abs(ref)
        bad = np.abs(go[t] - ref) > tol + half * (1 + 2.0 ** -7)
        assert not bad.any(), (t, int(bad.sum()), float(np.abs(go[t] - ref).max()), float(tol.max()))
        if with_lse:
            if len(sel) == 0:
                assert np.all(np.isneginf(gl[t])) and np.all(go[t] == 0)
            else:
                assert np.all(np.abs(gl[t] - rl) <= tl), (t, float(np.abs(gl[t] - rl).max()), float(tl.max()))
    return out, lse


ATTN = [
    # lens, per, page, H, k, tail, out
    ([50], [1], 0, 1, 1, True, "f32"),
    ([50], [1], 0, 64, 33, True, "bf16"),
    ([1], [1], 0, 8, 16, True, "f32"),                       # a sequence of one token
    ([3000, 2100], [1, 1], 0, 64, 2048, True, "bf16"),       # split decode
    ([3000, 700, 129], [1, 1, 1], 64, 128, 257, True, "f32"),
    ([500, 129, 1000], [1, 1, 1], 16, 40, 100, False, "f32"),
    ([700, 300], [130, 100], 0, 16, 384, True, "f32"),       # prefill: one CTA walks a token's tiles
    ([700, 300], [130, 100], 1, 65, 300, False, "bf16"),
    ([2100] * 20, [1] * 20, 64, 33, 2051, False, "bf16"),
    ([700, 300], [290, 200], 0, 70, 100, True, "bf16"),      # units of one tile, several per CTA
    ([700, 300], [290, 200], 4, 64, 128, False, "f32"),
    ([900, 300], [400, 200], 0, 64, 256, True, "f32"),       # of two
]


@pytest.mark.parametrize("lens,per,page,H,k,tail,out", ATTN)
def test_attention(dsa, torch, lens, per, page, H, k, tail, out):
    s = Seqs(dsa, torch, lens, per, page, seed=k)
    idx = selections(s, k, twice=True)
    T = len(s.pos)
    attend(dsa, torch, s, H, k, idx, tail, out_dt=out, check=range(0, T, max(1, T // 12)))


def test_attention_masks(dsa, torch):
    """-1 anywhere in a row, whole tiles of it, a row without any entry, one entry at the end."""
    s = Seqs(dsa, torch, [900], [160])
    idx = selections(s, 600)
    idx[3, ::4] = -1
    idx[4, :] = -1
    idx[5, :599] = -1
    idx[5, 599] = 700
    idx[6, 100:400] = -1
    idx[7, 1:] = -1
    attend(dsa, torch, s, 24, 600, idx, check=[0, 3, 4, 5, 6, 7, 159])


def test_attention_masks_in_split_decode(dsa, torch):
    s = Seqs(dsa, torch, [4000, 4000, 4000], [1, 1, 1])
    idx = selections(s, 2048)
    idx[0, :1500] = -1
    idx[1, :] = -1
    idx[2, 1:] = -1
    attend(dsa, torch, s, 64, 2048, idx, out_dt="bf16")


@pytest.mark.parametrize("spread,size", [(0.0, 30.0), (4.0, 1.0), (8.0, 0.01), (0.5, 1e-4)])
def test_attention_sharp_flat_and_uneven(dsa, torch, spread, size):
    """Sharp softmaxes that move the running maximum, rows whose scales differ
    by many powers of two, all but equal scores."""
    s = Seqs(dsa, torch, [1300], [155])
    attend(dsa, torch, s, 20, 700, selections(s, 700), spread=spread, size=size, check=range(0, 155, 31))
    d = Seqs(dsa, torch, [3000, 2500], [1, 1])
    attend(dsa, torch, d, 64, 2048, selections(d, 2048), spread=spread, size=size)


def test_attention_ascending_scores(dsa, torch):
    """The largest score grows from tile to tile: every tile raises the maximum."""
    s = Seqs(dsa, torch, [1000], [153])
    codes, scale = fill_cache(dsa, torch, s, False, 0.0)
    b = dsa.Batch.from_host([0, s.rows], range(s.rows), [0], s.rows)
    x = torch.randn(s.rows, 512, generator=gen(torch, 2), device="cuda") * 0.05
    x[:, 0] = torch.arange(s.rows, device="cuda") / 20.0
    dsa.dsa_kv_append_q8(x, None, b, None, codes, scale, s.ws)
    q = torch.zeros(153, 5, 512, device="cuda")
    q[:, :, 0] = torch.tensor([20.0, 3.0, 0.5, -3.0, 0.0], device="cuda")
    q = q.to(torch.bfloat16)
    idx = torch.from_numpy(selections(s, 640)).cuda()
    ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=5, k=640)
    out, lse = torch.empty(153, 5, 512, device="cuda"), torch.empty(153, 5, device="cuda")
    dsa.dsa_sparse_mla_attn_q8(q, None, codes, scale, s.batch, idx, 1.0, out, lse, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    c, sc, ix = codes.cpu().numpy(), f64(scale), idx.cpu().numpy()
    for t in (0, 76, 152):
        ref, rl, tol, tl = R.attention(f64(q[t]), None, c, sc, ix[t][ix[t] >= 0], 1.0)
        assert np.all(np.abs(f64(out[t]) - ref) <= tol)
        assert np.all(np.abs(f64(lse[t]) - rl) <= tl)


def test_attention_indices_out_of_range_are_skipped_and_flagged(dsa, torch):
    s = Seqs(dsa, torch, [300], [2])
    codes, scale = fill_cache(dsa, torch, s, True)
    idx = selections(s, 64)
    dirty = idx.copy()
    idx[0, [3, 10, 63]] = -1
    dirty[0, [3, 10, 63]] = [300, -2, 2 ** 31 - 1]
    q = torch.randn(2, 7, 512, device="cuda").to(torch.bfloat16)
    qr = torch.randn(2, 7, 64, device="cuda").to(torch.bfloat16)
    res = []
    for ix, want in ((idx, 0), (dirty, dsa.DSA_DEV_BAD_INDEX)):
        ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=7, k=64)
        out = torch.empty(2, 7, 512, device="cuda")
        dsa.dsa_sparse_mla_attn_q8(q, qr, codes, scale, s.batch, torch.from_numpy(ix).cuda(), 0.1, out, None, ws)
        assert dsa.dsa_read_device_status(ws) == want
        res.append(out)
    assert torch.equal(res[0], res[1])


def test_attention_ignores_garbage_in_rows_it_does_not_select(dsa, torch):
    """NaN codes and scales, infinities: in every unselected row, the query's own among them."""
    s = Seqs(dsa, torch, [2500], [1])
    codes, scale = fill_cache(dsa, torch, s, True)
    idx = selections(s, 500)
    idx[idx == 2499] = -1
    idx[0, 77] = -1
    q = torch.randn(1, 64, 512, device="cuda").to(torch.bfloat16)
    qr = torch.randn(1, 64, 64, device="cuda").to(torch.bfloat16)
    ix = torch.from_numpy(idx).cuda()
    res = []
    for dirty in (False, True):
        if dirty:
            rest = torch.ones(s.rows, dtype=torch.bool, device="cuda")
            rest[ix[ix >= 0].long()] = False
            codes[rest] = 0x7F
            scale[rest] = float("nan")
            scale[rest.nonzero()[::2, 0]] = float("inf")
        ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=64, k=500)
        out, lse = torch.empty(1, 64, 512, device="cuda"), torch.empty(1, 64, device="cuda")
        dsa.dsa_sparse_mla_attn_q8(q, qr, codes, scale, s.batch, ix, 0.05, out, lse, ws)
        res.append((out, lse))
    assert torch.isfinite(res[1][0]).all()
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_calls_repeat_bit_for_bit_on_streams_and_in_a_graph(dsa, torch):
    """Append, read and attention on a side stream and replayed from a graph
    with new inputs in the same buffers."""
    s = Seqs(dsa, torch, [1500, 900], [1, 1], 64)
    codes, scale = fill_cache(dsa, torch, s, True)
    rope = dsa.Rope.make(64, 1e4, True)
    c_new = torch.randn(2, 576, device="cuda").to(torch.bfloat16)
    q_in = torch.randn(2, 64, 576, device="cuda").to(torch.bfloat16)
    idx = torch.from_numpy(selections(s, 512)).cuda()
    idx[0, -1], idx[1, -1] = 1499, 899
    ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=64, k=512)
    q_lat, q_rope = q_in[:, :, :512].contiguous(), torch.empty(2, 64, 64, dtype=torch.bfloat16, device="cuda")

    def step(out, lse, back):
        dsa.dsa_rope(q_in[:, :, 512:], s.batch.q_pos, rope, q_rope)
        dsa.dsa_kv_append_q8(c_new[:, :512], c_new[:, 512:], s.batch, rope, codes, scale, ws, *s.paging)
        dsa.dsa_sparse_mla_attn_q8(q_lat, q_rope, codes, scale, s.batch, idx, 0.07, out, lse, ws, *s.paging)
        dsa.dsa_kv_read_q8(codes, scale, s.batch, back, ws, *s.paging)

    def buffers():
        return (torch.empty(2, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 64, device="cuda"),
                torch.empty(2, 576, dtype=torch.bfloat16, device="cuda"))

    first = buffers()
    step(*first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side, graphed = buffers(), buffers()
    with torch.cuda.stream(side):
        step(*on_side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*graphed)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, on_side, graphed):
        assert torch.equal(a, b) and torch.equal(a, c)
    c_new.copy_(torch.randn(2, 576, device="cuda"))
    graph.replay()
    again = buffers()
    step(*again)
    torch.cuda.synchronize()
    for a, b in zip(again, graphed):
        assert torch.equal(a, b)
    assert not torch.equal(again[2], first[2])
    assert dsa.dsa_read_device_status(ws) == 0


def test_tensors_on_the_host_are_refused(dsa, torch):
    s = Seqs(dsa, torch, [9], [1])
    codes, scale = dsa.q8_cache(s.rows)
    x = torch.randn(1, 576)
    with pytest.raises(TypeError):
        dsa.dsa_kv_append_q8(x[:, :512], x[:, 512:], s.batch, None, codes, scale, s.ws)
    with pytest.raises(TypeError):
        dsa.dsa_kv_read_q8(codes.cpu(), scale, s.batch, x.cuda(), s.ws)
    with pytest.raises(TypeError):
        dsa.dsa_rope(x[None], torch.zeros(1, dtype=torch.int32), dsa.Rope.make(64), x[None])


@pytest.mark.parametrize("lens,per,k", [([700], [400], 600), ([3000, 2500], [1, 1], 2048)])
def test_attention_waits_that_run_out(dsa, torch, lens, per, k):
    """Producers that copy nothing (the failure-path hook): the call reports
    DSA_DEV_TIMEOUT, and the next one is right again."""
    s = Seqs(dsa, torch, lens, per)
    idx = selections(s, k)
    codes, scale = fill_cache(dsa, torch, s, True)
    T = s.batch.T
    q = torch.randn(T, 8, 512, device="cuda").to(torch.bfloat16)
    qr = torch.randn(T, 8, 64, device="cuda").to(torch.bfloat16)
    ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=8, k=k)
    out = torch.empty(T, 8, 512, device="cuda")
    args = (q, qr, codes, scale, s.batch, torch.from_numpy(idx).cuda(), 0.1, out, None, ws)
    try:
        dsa.dsa_set_test_faults(wait_limit_ns=2_000_000, skip_copies=True)
        dsa.dsa_sparse_mla_attn_q8(*args)
        assert dsa.dsa_read_device_status(ws) & dsa.DSA_DEV_TIMEOUT
    finally:
        dsa.dsa_set_test_faults()
    attend(dsa, torch, s, 8, k, idx, check=[0, T - 1])


def test_attention_many_units(dsa, torch):
    """Several thousand units of different lengths, bad positions among them:
    CTAs take over units of CTAs that have not started."""
    s = Seqs(dsa, torch, [3000, 900], [2900, 850])
    k = 200
    idx = selections(s, k)
    idx[::7] = -1
    codes, scale = fill_cache(dsa, torch, s, True)
    pos = s.batch.q_pos.clone()
    pos[5::11] = -1
    s.batch.q_pos = pos
    H = 3
    q = torch.randn(s.batch.T, H, 512, device="cuda").to(torch.bfloat16)
    qr = torch.randn(s.batch.T, H, 64, device="cuda").to(torch.bfloat16)
    ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=H, k=k)
    out = torch.full((s.batch.T, H, 512), float("nan"), device="cuda")
    lse = torch.full((s.batch.T, H), float("nan"), device="cuda")
    dsa.dsa_sparse_mla_attn_q8(q, qr, codes, scale, s.batch, torch.from_numpy(idx).cuda(), 0.1, out, lse, ws)
    assert dsa.dsa_read_device_status(ws) == dsa.DSA_DEV_BAD_POSITION
    go, gl, c, sc = f64(out), f64(lse), codes.cpu().numpy(), f64(scale)
    empty = np.zeros(len(s.pos), bool)
    empty[::7] = True
    empty[5::11] = True
    assert np.all(go[empty] == 0) and np.all(np.isneginf(gl[empty]))
    assert np.all(np.isfinite(go[~empty])) and np.all(np.isfinite(gl[~empty]))
    for t in np.nonzero(~empty)[0][::97]:
        rows = np.asarray(s.row(int(s.seq[t]), idx[t][idx[t] >= 0]))
        ref, rl, tol, tl = R.attention(f64(q[t]), f64(qr[t]), c, sc, rows, 0.1)
        assert np.all(np.abs(go[t] - ref) <= tol * (1 + 2.0 ** -7) + 2.0 ** -24) and np.all(np.abs(gl[t] - rl) <= tl)


def test_decode_step_over_the_8_bit_cache(dsa, torch):
    """A whole step as a server runs it: the indexer's keys, scores and top-k,
    the new tokens' rows turned and appended, their queries turned, attention
    over the selection; against 64 bits over the cache and selection it left."""
    lens, H, H_I, k = [2900, 1200, 300], 64, 32, 512
    s = Seqs(dsa, torch, lens, [1, 1, 1])
    codes, scale = fill_cache(dsa, torch, s, True)
    before = codes.clone()
    g = gen(torch, 21)
    keys = torch.randn(s.rows, 128, generator=g, device="cuda").half()
    k_new = torch.randn(3, 128, generator=g, device="cuda").half()
    q_idx = torch.randn(3, H_I, 128, generator=g, device="cuda").half()
    w = torch.rand(3, H_I, generator=g, device="cuda")
    c_new = torch.randn(3, 512, generator=g, device="cuda").to(torch.bfloat16)
    r_new = torch.randn(3, 64, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(3, H, 576, generator=g, device="cuda").to(torch.bfloat16)
    rope = dsa.Rope.make(64, 1e4, True, "yarn", 4.0, 1024)
    idx = torch.empty(3, k, dtype=torch.int32, device="cuda")
    width = (max(lens) + 127) // 128 * 128
    scores = torch.empty(3, width, device="cuda")
    out, lse = torch.empty(3, H, 512, device="cuda"), torch.empty(3, H, device="cuda")
    ws = {op: dsa.workspace(op, s.batch, H_I, H, k) for op in (dsa.DSA_OP_K_APPEND, dsa.DSA_OP_INDEXER_SCORE,
                                                               dsa.DSA_OP_TOPK, dsa.DSA_OP_SPARSE_ATTN)}
    dsa.dsa_indexer_k_append(k_new, s.batch, keys, False, ws[dsa.DSA_OP_K_APPEND])
    dsa.dsa_kv_append_q8(c_new, r_new, s.batch, rope, codes, scale, ws[dsa.DSA_OP_K_APPEND])
    dsa.dsa_indexer_score(q_idx, w, keys, s.batch, False, scores, ws[dsa.DSA_OP_INDEXER_SCORE])
    dsa.dsa_topk(scores, s.batch, k, idx, ws[dsa.DSA_OP_TOPK])
    dsa.dsa_rope(q, s.batch.q_pos, rope, q, 512)
    q_lat, q_rope = q[:, :, :512].contiguous(), q[:, :, 512:].contiguous()
    dsa.dsa_sparse_mla_attn_q8(q_lat, q_rope, codes, scale, s.batch, idx, 0.07, out, lse, ws[dsa.DSA_OP_SPARSE_ATTN])
    assert all(dsa.dsa_read_device_status(v) == 0 for v in ws.values())
    at = torch.from_numpy(s.token_rows()).cuda()
    others = torch.ones(s.rows, dtype=torch.bool, device="cuda")
    others[at] = False
    assert torch.equal(codes[others], before[others]) and not torch.equal(codes[at], before[at])
    c, sc, sel = codes.cpu().numpy(), f64(scale), idx.cpu().numpy()
    for t in range(3):
        mine = sel[t][sel[t] >= 0]
        assert len(mine) == min(k, lens[t])
        ref, rl, tol, tl = R.attention(f64(q_lat[t]), f64(q_rope[t]), c, sc, np.asarray(s.row(t, mine)), 0.07)
        assert np.all(np.abs(f64(out[t]) - ref) <= tol) and np.all(np.abs(f64(lse[t]) - rl) <= tl)


def test_two_streams_at_once(dsa, torch):
    """Two attention calls side by side, each with its own workspace, give what
    they give alone: split decodes and a grid of several waves."""
    def setup(s, H, k, seed):
        codes, scale = fill_cache(dsa, torch, s, True, seed=seed)
        g = gen(torch, seed + 1)
        T = s.batch.T
        q = torch.randn(T, H, 512, generator=g, device="cuda").to(torch.bfloat16)
        r = torch.randn(T, H, 64, generator=g, device="cuda").to(torch.bfloat16)
        idx = torch.from_numpy(selections(s, k, seed)).cuda()
        ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=H, k=k)

        def call():
            out, lse = torch.empty(T, H, 512, device="cuda"), torch.empty(T, H, device="cuda")
            dsa.dsa_sparse_mla_attn_q8(q, r, codes, scale, s.batch, idx, 0.06, out, lse, ws, *s.paging)
            return out, lse
        return call, ws

    calls = [setup(Seqs(dsa, torch, [3000, 2500, 600], [1, 1, 1]), 64, 2048, 31),
             setup(Seqs(dsa, torch, [900, 500], [200, 150], 16), 128, 300, 41)]
    alone = [c() for c, _ in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(4):
        got = []
        for (c, _), st in zip(calls, streams):
            with torch.cuda.stream(st):
                got.append(c())
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(dsa.dsa_read_device_status(ws) == 0 for _, ws in calls)


def test_calls_in_a_row_see_what_the_one_before_wrote(dsa, torch):
    """The calls start while what precedes them ends: a hundred rounds without a
    pause of torch kernel -> append -> read -> rotation in place and back ->
    attention over the row just written, eager and from a graph in which
    copies, a memset and a joined side stream precede them."""
    B, H = 5, 16
    s = Seqs(dsa, torch, [40] * B, [1] * B)
    codes, scale = dsa.q8_cache(s.rows)
    ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=H, k=1)
    idx = torch.full((B, 1), 39, dtype=torch.int32, device="cuda")        # its own row: the output is that row
    c_new, r_new = (torch.zeros(B, n, dtype=torch.bfloat16, device="cuda") for n in (512, 64))
    q, qr = (torch.ones(B, H, n, dtype=torch.bfloat16, device="cuda") for n in (512, 64))
    back = torch.empty(B, 576, device="cuda")
    out = torch.empty(B, H, 512, device="cuda")
    rope = dsa.Rope.make(64, 1e4, False)
    x = torch.empty(B, H, 64, device="cuda")
    rounds = [(-1) ** i * 2.0 ** (i % 13) for i in range(100)]           # e4m3 holds them exactly
    got = torch.empty(len(rounds), 3, device="cuda")

    def calls():
        dsa.dsa_kv_append_q8(c_new, r_new, s.batch, None, codes, scale, ws)
        dsa.dsa_kv_read_q8(codes, scale, s.batch, back, ws)
        dsa.dsa_rope(x, s.batch.q_pos, rope, x)
        dsa.dsa_rope(x, s.batch.q_pos, rope, x, inverse=True)
        dsa.dsa_sparse_mla_attn_q8(q, qr, codes, scale, s.batch, idx, 0.01, out, None, ws)

    def check(tol=2.0 ** -20):
        g = got.cpu().numpy()
        for i, v in enumerate(rounds):
            assert g[i, 0] == v and g[i, 1] == v, (i, v, g[i])
            assert abs(g[i, 2] - v) <= tol * 4 * abs(v), (i, v, g[i])

    def note(i):
        got[i, 0], got[i, 1] = back.amin(), out.amin()
        got[i, 2] = x.amin() if rounds[i] > 0 else x.amax()

    for i, v in enumerate(rounds):
        c_new.fill_(v)
        r_new.fill_(v)
        x.fill_(v)
        calls()
        note(i)
    torch.cuda.synchronize()
    check()
    src = torch.zeros(B, 512, dtype=torch.bfloat16, device="cuda")
    val = torch.zeros((), device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            r_new.copy_(src[:, :64])
            x.copy_(val.expand(B, H, 64))
        codes.zero_()                                                     # a memset
        main.wait_stream(side)
        c_new.copy_(src)                                                  # a copy
        calls()
    got.zero_()
    for i, v in enumerate(rounds):
        src.fill_(v)
        val.fill_(v)
        graph.replay()
        note(i)
    torch.cuda.synchronize()
    check()
    assert dsa.dsa_read_device_status(ws) == 0


@pytest.mark.parametrize("seed", range(4))
def test_attention_shapes_drawn(dsa, torch, seed):
    """Lengths, new tokens, pages, heads, selections, masks and orders drawn at random."""
    rng = np.random.default_rng(900 + seed)
    for _ in range(12):
        B = int(rng.choice([1, 2, 5]))
        lens = [int(n) for n in rng.choice([1, 2, 127, 128, 129, 500, 1500], B)]
        per = [min(n, int(rng.choice([1, 3, 130, 260]))) for n in lens]
        k, H = int(rng.choice([1, 100, 128, 129, 256, 385, 1000])), int(rng.choice([1, 8, 33, 64, 65, 128]))
        s = Seqs(dsa, torch, lens, per, int(rng.choice([0, 1, 16, 64])), seed=int(rng.integers(1000)))
        idx = selections(s, k, seed=int(rng.integers(1000)))
        idx[rng.random(idx.shape) < rng.choice([0.0, 0.3, 0.95])] = -1
        idx = np.ascontiguousarray(idx[:, rng.permutation(k)])
        T = len(s.pos)
        attend(dsa, torch, s, H, k, idx, bool(rng.random() < 0.6), out_dt=["f32", "bf16"][int(rng.integers(2))],
               check=sorted({0, T - 1, int(rng.integers(T))}))
