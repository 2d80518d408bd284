"""The 8-bit attention, its cache and the rotation where they can go wrong:
tails alone deciding the scores, rows and queries that are not finite, far
scales, the spread of the errors; against float64 (tests/_q8_ref.py, which
derives the bounds that are not derived here)."""
import numpy as np
import pytest

import _q8_ref as R
from test_gpu_q8 import Seqs, dsa, f64, fill_cache, gen, selections, torch  # noqa: F401  (two fixtures among them)

pytestmark = pytest.mark.gpu


def attend(dsa, torch, s, q, qr, codes, scale, idx, sm, out_dt=None):
    """(out, lse) of one call, its status checked."""
    T, H, k = q.shape[0], q.shape[1], idx.shape[1]
    ws = dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, s.batch, H=H, k=k)
    out = torch.full((T, H, 512), -7.0, dtype=out_dt or torch.float32, device="cuda")
    lse = torch.full((T, H), -7.0, device="cuda")
    ix = torch.from_numpy(idx).cuda() if isinstance(idx, np.ndarray) else idx
    dsa.dsa_sparse_mla_attn_q8(q, qr, codes, scale, s.batch, ix, sm, out, lse, ws, *s.paging)
    assert dsa.dsa_read_device_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("lens,per,k", [([2300], [160], 2048), ([1500, 900], [200, 140], 700)])
def test_scores_of_the_tails_alone(dsa, torch, lens, per, k):
    """Latent queries of zero: every score is its row's tail, whose place in
    tensor memory is written again two tiles later (6 to 16 tiles a token,
    several tokens a CTA)."""
    s = Seqs(dsa, torch, lens, per)
    codes, scale = fill_cache(dsa, torch, s, True, 0.0)
    T, H, sm = s.batch.T, 64, 0.5
    q = torch.zeros(T, H, 512, dtype=torch.bfloat16, device="cuda")
    qr = torch.randn(T, H, 64, generator=gen(torch, 3), device="cuda").to(torch.bfloat16)
    idx = selections(s, k)
    first = attend(dsa, torch, s, q, qr, codes, scale, idx, sm)
    c, sc = codes.cpu().numpy(), f64(scale)
    for t in range(0, T, 23):
        rows = np.asarray(s.row(int(s.seq[t]), idx[t][idx[t] >= 0]))
        ref, rl, tol, tl = R.attention(f64(q[t]), f64(qr[t]), c, sc, rows, sm)
        assert np.all(np.abs(f64(first[0][t]) - ref) <= tol) and np.all(np.abs(f64(first[1][t]) - rl) <= tl)
    for _ in range(20):
        again = attend(dsa, torch, s, q, qr, codes, scale, idx, sm)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("heads_first", [False, True])
def test_rotation_between_slices_of_one_buffer(dsa, torch, heads_first):
    """Parts of the same heads and groups of heads, packed as tightly as they are taken."""
    T, H = 5, 6
    rope = dsa.Rope.make(64, 1e4, False)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    for parts in (True, False):
        shape = (T, H, 2, 64) if parts else (T, 2, H, 64)
        buf = torch.randn(shape, generator=gen(torch, 4), device="cuda").to(torch.bfloat16)
        if heads_first:
            buf = torch.randn((H,) + ((T, 2, 64) if parts else (2, T, 64)), generator=gen(torch, 4), device="cuda").to(torch.bfloat16)
        a, b = (buf.select(2 if parts else 1, i) for i in (0, 1))
        if heads_first:
            a, b = a.transpose(0, 1), b.transpose(0, 1)
        for x, y in ((a, b), (b, a)):
            keep, want = x.clone(), torch.empty_like(x, memory_format=torch.contiguous_format)
            dsa.dsa_rope(keep, pos, rope, want)
            dsa.dsa_rope(x, pos, rope, y)
            assert torch.equal(y, want) and torch.equal(x, keep)


def test_rotation_of_a_long_head_major_view(dsa, torch):
    """Heads 131072 tokens of 128 values apart, in place: the bits of the packed call."""
    T, H, D = 131072, 2, 128
    x = torch.randn(H, T, D, generator=gen(torch, 6), device="cuda").to(torch.bfloat16).transpose(0, 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rope = dsa.Rope.make(64, 1e6, True, "yarn", 4.0, 32768)
    want = torch.empty(T, H, D, dtype=x.dtype, device="cuda")
    dsa.dsa_rope(x.contiguous(), pos, rope, want, 64)
    dsa.dsa_rope(x, pos, rope, x, 64)
    assert torch.equal(x, want)


def test_rotation_in_place_of_one_token_whatever_its_stride(dsa, torch):
    rope = dsa.Rope.make(64, 1e4, True)
    pos = torch.tensor([77], dtype=torch.int32, device="cuda")
    x = torch.randn(1, 8, 64, generator=gen(torch, 6), device="cuda")
    want = torch.empty_like(x)
    dsa.dsa_rope(x, pos, rope, want)
    dsa.dsa_rope(x, pos, rope, x.as_strided((1, 8, 64), (3, 64, 1)))
    assert torch.equal(x, want)


NOT_FINITE = [
    # lens, per, k: split (one token each of two sequences) and one CTA per token
    ([2600, 1300], [1, 1], 1024),
    ([1300], [160], 300),
]


def not_finite_case(dsa, torch, lens, per, k, tail, seed=13):
    s = Seqs(dsa, torch, lens, per)
    codes, scale = fill_cache(dsa, torch, s, tail)
    g = gen(torch, seed)
    q = torch.randn(s.batch.T, 70, 512, generator=g, device="cuda").to(torch.bfloat16)
    qr = torch.randn(s.batch.T, 70, 64, generator=g, device="cuda").to(torch.bfloat16) if tail else None
    return s, codes, scale, q, qr


@pytest.mark.parametrize("lens,per,k", NOT_FINITE)
@pytest.mark.parametrize("tail", [True, False])
def test_selected_rows_that_are_not_finite(dsa, torch, lens, per, k, tail):
    """Rows with the scale NaN, as the append leaves them: among finite ones,
    alone, alone in a tile, beside masked ones.  Out and lse are NaN where one
    is selected and untouched where none is."""
    s, codes, scale, q, qr = not_finite_case(dsa, torch, lens, per, k, tail)
    idx = selections(s, k)
    good = attend(dsa, torch, s, q, qr, codes, scale, idx, 0.05)
    last = s.batch.T - 1                                   # the first tokens stay as they are
    at = int(idx[last][k // 3])
    x = torch.full((1, 576 if tail else 512), float("inf"), device="cuda")
    one = dsa.Batch.from_host([0, 1], [at], [s.off[int(s.seq[last])]], s.rows)
    dsa.dsa_kv_append_q8(x[:, :512], x[:, 512:] if tail else None, one, None, codes, scale, s.ws)
    only = np.full_like(idx[last], -1)
    for how in range(5):
        ix = idx.copy()
        if how == 1:
            ix[last], ix[last, 0] = -1, at                 # alone, first
        elif how == 2:
            ix[last], ix[last, -1] = -1, at                # alone, in the last tile
        elif how == 3:
            ix[last] = at                                  # nothing else, all through
        elif how == 4:
            ix[last] = only                                # none
        hit = (ix == at).any(1) & (s.seq == s.seq[last])
        for dt in (torch.float32, torch.bfloat16):
            out, lse = attend(dsa, torch, s, q, qr, codes, scale, ix, 0.05, dt)
            for t in range(s.batch.T):
                if hit[t]:
                    assert torch.isnan(out[t]).all() and torch.isnan(lse[t]).all(), (how, t)
                elif t == last:
                    assert (out[t] == 0).all() and torch.isneginf(lse[t]).all(), (how, t)
                else:
                    assert torch.equal(out[t], good[0][t].to(dt)) and torch.equal(lse[t], good[1][t]), (how, t)


@pytest.mark.parametrize("lens,per,k", NOT_FINITE)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_queries_that_are_not_finite(dsa, torch, lens, per, k, bad):
    """One head's query: that head alone is lost, and only where rows are
    selected; the first tiles of a token fully masked as well."""
    s, codes, scale, q, qr = not_finite_case(dsa, torch, lens, per, k, True)
    idx = selections(s, k)
    idx[0, :k // 2] = -1
    idx[-1] = -1
    sm = 4.0                                               # (references far from the first tile's)
    good = attend(dsa, torch, s, q, qr, codes, scale, idx, sm)
    assert (good[0][-1] == 0).all() and torch.isneginf(good[1][-1]).all()
    q[:, 5, 100] = bad
    qr[:, 67, 3] = bad
    out, lse = attend(dsa, torch, s, q, qr, codes, scale, idx, sm)
    lost = torch.zeros(s.batch.T, 70, dtype=torch.bool, device="cuda")
    lost[:-1, 5] = lost[:-1, 67] = True
    assert torch.isnan(out[lost]).all() and torch.isnan(lse[lost]).all()
    assert torch.equal(out[~lost], good[0][~lost]) and torch.equal(lse[~lost], good[1][~lost])


def test_paged_calls_do_not_read_the_sequences_offsets(dsa, torch):
    """With a block table kv_off may hold anything: every paged call gives what
    it gives over zeros."""
    s = Seqs(dsa, torch, [700, 300], [3, 2], 64)
    codes0, scale0 = fill_cache(dsa, torch, s, True)
    idx = torch.from_numpy(selections(s, 200)).cuda()
    g = gen(torch, 8)
    q = torch.randn(5, 16, 512, generator=g, device="cuda").to(torch.bfloat16)
    qr = torch.randn(5, 16, 64, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn(5, 576, generator=g, device="cuda").to(torch.bfloat16)
    keys0 = torch.randn(s.rows, 128, generator=g, device="cuda").half()
    k_new = torch.randn(5, 128, generator=g, device="cuda").half()
    q_idx = torch.randn(5, 32, 128, generator=g, device="cuda").half()
    w = torch.rand(5, 32, generator=g, device="cuda")
    kv = torch.randn(s.rows, 576, generator=g, device="cuda").to(torch.bfloat16)
    got = []
    for off in ([0, 0], [-7, 1 << 40]):
        s.batch.kv_off = torch.tensor(off, dtype=torch.int64, device="cuda")
        codes, scale, keys, cache = codes0.clone(), scale0.clone(), keys0.clone(), kv.clone()
        dsa.dsa_kv_append_q8(x[:, :512], x[:, 512:], s.batch, None, codes, scale, s.ws, *s.paging)
        dsa.dsa_kv_append(x[:, :512], x[:, 512:], s.batch, None, cache, s.ws, *s.paging)
        back = torch.empty(5, 576, device="cuda")
        dsa.dsa_kv_read_q8(codes, scale, s.batch, back, s.ws, *s.paging)
        assert dsa.dsa_read_device_status(s.ws) == 0
        o8 = attend(dsa, torch, s, q, qr, codes, scale, idx, 0.07)
        ws = dsa.workspace(dsa.DSA_OP_DECODE, s.batch, 32, 16, 200)
        out, lse = torch.empty(5, 16, 512, device="cuda"), torch.empty(5, 16, device="cuda")
        sel = torch.empty(5, 200, dtype=torch.int32, device="cuda")
        dsa.dsa_decode_paged(k_new, q_idx, w, q, qr, keys, cache, s.batch, s.block, 64, 200, 0.07, False, out, lse, sel, ws)
        assert dsa.dsa_read_device_status(ws) == 0
        got.append((codes, scale, cache, back, *o8, keys, out, lse, sel))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def pi(digits=60):
    """pi by Machin's formula."""
    from decimal import Decimal, getcontext
    getcontext().prec = digits + 10

    def arctan_inv(n):
        total = term = Decimal(1) / n
        k = 1
        while abs(term) > Decimal(10) ** -(digits + 5):
            term /= -n * n
            k += 2
            total += term / k
        return total
    return 16 * arctan_inv(5) - 4 * arctan_inv(239)


def test_angles_of_far_positions_and_of_any_frequency(dsa, torch):
    """Against exact products: the turn is off by less than (|f| + 1) |p| 2^-64
    and the 2^-32 its fraction is cut to, then rounded (2^-25 of a turn); the
    sine and cosine add two units of 2^-24."""
    from decimal import Decimal
    f = [0.0, 1e-30, 2.0 ** -60, 1e-12, 1e-4, 0.7, 1.0, -1.0, -3.1, 1000.0, 2.0 ** 20, 12345.678]
    two_pi = 2 * pi()
    pos = [0, 1, -1, 4097, 1 << 20, 2 ** 31 - 1, -2 ** 31]
    rope = dsa.Rope(torch.tensor(f, dtype=torch.float64, device="cuda"), True)
    x = torch.zeros(len(pos), 1, 2 * len(f), device="cuda")
    x[:, :, 0::2] = 1.0
    y = torch.empty_like(x)
    dsa.dsa_rope(x, torch.tensor(pos, dtype=torch.int32, device="cuda"), rope, y)
    got = f64(y)[:, 0]
    for i, p in enumerate(pos):
        for j, v in enumerate(f):
            turn = float((Decimal(p) * Decimal(v) / two_pi) % 1)
            tol = 2 * np.pi * ((abs(v) + 1) * abs(p) * 2.0 ** -64 + 2.0 ** -32 + 2.0 ** -25) + 2.0 ** -23
            assert abs(got[i, 2 * j] - np.cos(2 * np.pi * turn)) <= tol, (p, v)
            assert abs(got[i, 2 * j + 1] - np.sin(2 * np.pi * turn)) <= tol, (p, v)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("inter", [True, False])
def test_frequencies_that_are_not_finite_give_nan(dsa, torch, bad, inter):
    s = Seqs(dsa, torch, [50], [4])
    rope, wrong = dsa.Rope.make(64, 1e4, inter), dsa.Rope.make(64, 1e4, inter)
    wrong.inv_freq[5] = bad
    x = torch.randn(4, 576, generator=gen(torch, 8), device="cuda")
    hit = torch.zeros(64, dtype=torch.bool, device="cuda")
    hit[[10, 11] if inter else [5, 37]] = True
    want, got = torch.empty(4, 1, 64, device="cuda"), torch.empty(4, 1, 64, device="cuda")
    dsa.dsa_rope(x[:, None, 512:], s.batch.q_pos, rope, want)
    dsa.dsa_rope(x[:, None, 512:], s.batch.q_pos, wrong, got)
    assert torch.isnan(got[..., hit]).all() and torch.equal(got[..., ~hit], want[..., ~hit])
    kv = torch.zeros(s.rows, 576, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_kv_append(x[:, :512], x[:, 512:], s.batch, wrong, kv, s.ws)
    new = kv[torch.from_numpy(s.token_rows()).cuda()]
    assert torch.isnan(new[:, 512:][:, hit]).all() and torch.isfinite(new[:, 512:][:, ~hit]).all()
    codes, scale = dsa.q8_cache(s.rows)
    dsa.dsa_kv_append_q8(x[:, :512], x[:, 512:], s.batch, wrong, codes, scale, s.ws)
    assert torch.isnan(scale[torch.from_numpy(s.token_rows()).cuda()]).all()


def test_sines_and_cosines_to_their_last_bit(dsa, torch):
    """x = (1, 0) turned: float32 sine and cosine of pi times the fraction are
    good to a unit of 2^-24, what the rounded fraction left out is put back to
    2^-32 of a turn (and C, F and their product to less), and that sum is
    rounded once more.  A fraction rounded to 24 bits alone would be off by up
    to 2 pi 2^-26 by itself, as much as all of that."""
    T = 3000
    f, _ = dsa.dsa_rope_frequencies(64, 10000.0)
    rope = dsa.Rope(torch.tensor(f, dtype=torch.float64, device="cuda"), True)
    pos = torch.randint(0, 1 << 18, (T,), generator=gen(torch, 5), device="cuda", dtype=torch.int32)
    x = torch.zeros(T, 1, 64, device="cuda")
    x[:, :, 0::2] = 1.0
    y = torch.empty_like(x)
    dsa.dsa_rope(x, pos, rope, y)
    # 64 bits hold angles below 2^18 to 2^-36
    ang = pos.double()[:, None] * rope.inv_freq
    err = torch.maximum((y[:, 0, 0::2].double() - ang.cos()).abs(), (y[:, 0, 1::2].double() - ang.sin()).abs())
    assert float(err.max()) <= 2.0 ** -24 + 2.0 ** -25 + 2 * np.pi * 2.0 ** -31.9, float(err.max())


@pytest.mark.parametrize("lens,per,k", [([2600, 1300], [1, 1], 1024), ([900], [160], 300)])
@pytest.mark.parametrize("dq,drow,dsm", [(-60, 60, 0), (-100, 100, 0), (-100, 120, -20), (60, -25, -35)])
def test_small_queries_over_large_rows(dsa, torch, lens, per, k, dq, drow, dsm):
    """Queries times 2^dq, row scales times 2^drow, sm_scale times 2^dsm, summing
    to nothing: the same weights, outputs times 2^drow.  The pieces of the
    queries are the same; u = z log2 e + log2 scale is rounded twice at up to
    2^8 (2^-17 each, on both sides: 2^-15), and the weights anew, where their
    units lie otherwise: 2^-7 + 2^-11 of each on both sides, and 2^-14.9 of the
    largest; split partials by 2^-8."""
    s = Seqs(dsa, torch, lens, per)
    codes, scale = fill_cache(dsa, torch, s, True)
    g = gen(torch, 17)
    T, H, sm = s.batch.T, 33, 1 / 13.86
    q = torch.randn(T, H, 512, generator=g, device="cuda").to(torch.bfloat16)
    qr = torch.randn(T, H, 64, generator=g, device="cuda").to(torch.bfloat16)
    idx = selections(s, k)
    out0, lse0 = attend(dsa, torch, s, q, qr, codes, scale, idx, sm)
    out, lse = attend(dsa, torch, s, q * 2.0 ** dq, qr * 2.0 ** dq, codes, scale * 2.0 ** drow, idx, sm * 2.0 ** dsm)
    assert ((lse - lse0).abs() <= 2.0 ** -15 * (1 + lse0.abs())).all(), float((lse - lse0).abs().max())
    c, sc = codes.cpu().numpy(), f64(scale)
    for t in range(0, T, 13):
        rows = np.asarray(s.row(int(s.seq[t]), idx[t][idx[t] >= 0]))
        lat, tail = R.decode_rows(c[rows], sc[rows])
        z = sm * (f64(q[t]) @ lat.T + f64(qr[t]) @ tail.T)
        w = np.exp(z - f64(lse0[t])[:, None])
        top = (w * sc[rows]).max(1, keepdims=True)
        tol = (2 * (2.0 ** -7 + 2.0 ** -11) + 2 * 2.0 ** -8 + 2.0 ** -14) * (w @ np.abs(lat)) + \
            2 * 2.0 ** -14.9 * top * np.abs(lat / sc[rows][:, None]).sum(0)
        assert np.all(np.abs(f64(out[t]) * 2.0 ** -drow - f64(out0[t])) <= tol), t


RMS = [
    # lens, per, k, H: split decodes, then one CTA per token
    ([4000] * 3, [1] * 3, 2048, 64),
    ([4000, 3000], [1, 1], 600, 128),
    ([4000], [1], 100, 64),
    ([2500], [160], 2048, 16),
    ([1500], [160], 300, 16),
    ([1500], [160], 100, 16),
]


@pytest.mark.parametrize("lens,per,k,H", RMS)
@pytest.mark.parametrize("out_dt", ["f32", "bf16"])
def test_rms_error_of_the_outputs(dsa, torch, lens, per, k, H, out_dt):
    """Worst cases over all rows say little about errors that average out, so
    here their root mean square over everything, against the sum of squares of
    the outputs.  Rounding v in [1, 2) of a binade is off by
      an e4m3 piece and an e5m2 remainder: the first leaves an error uniform in
        +-2^-4, whose rounding is uniform in +-2^-3 of its own binade: a mean
        square of 2^-16 / 3 (1/2 + 1/16 + 1/128 ..) = 2^-16 / 3 * 4/7;
      bf16: 2^-16 / 3;  fp16 (weights before their pieces, split partials): 2^-22 / 3.
    v^2 is 3 / (2 ln 2) = 2.16 on average over weights spread over several
    octaves, and at least 1.8 over normal outputs whatever their size.  Rows of
    random signs add up in squares, so weights off by r leave outputs off by r.
    A tenth is allowed on top for the drawn sizes.  Without the weights' remainder
    the error is 4 to 16 times as large; partials in bf16 alone are off by
    2^-8 / sqrt(3 * 1.85) = 1.66e-3, the float32 bound is 1.32e-3."""
    s = Seqs(dsa, torch, lens, per)
    codes, scale = fill_cache(dsa, torch, s, True, 0.3)
    g = gen(torch, 19)
    T, sm = s.batch.T, 1 / 16.0
    q = torch.randn(T, H, 512, generator=g, device="cuda").to(torch.bfloat16)
    qr = torch.randn(T, H, 64, generator=g, device="cuda").to(torch.bfloat16)
    idx = selections(s, k)
    out, _ = attend(dsa, torch, s, q, qr, codes, scale, idx, sm, {"f32": torch.float32, "bf16": torch.bfloat16}[out_dt])
    c, sc = codes.cpu().numpy(), f64(scale)
    err = size = 0.0
    for t in range(0, T, 7 if T > 7 else 1):
        rows = np.asarray(s.row(int(s.seq[t]), idx[t][idx[t] >= 0]))
        ref = R.attention(f64(q[t]), f64(qr[t]), c, sc, rows, sm)[0]
        err += ((f64(out[t]) - ref) ** 2).sum()
        size += (ref ** 2).sum()
    weights, half, bf16 = 2.0 ** -16 / 3 * 4 / 7, 2.0 ** -22 / 3, 2.0 ** -16 / 3
    square = weights / 2.16 + 2 * half / 1.8 + (bf16 / 1.8 if out_dt == "bf16" else 0.0)
    print(f"\nrms {lens[0]} {T} {k} {out_dt}: {np.sqrt(err / size):.3e} of {np.sqrt(square):.3e}")
    assert np.sqrt(err / size) <= 1.1 * np.sqrt(square)


def test_split_partials_at_their_largest(dsa, torch):
    """Rows of the largest code throughout, and weights of nearly 2^8 in all but
    the first tile of each split (which sets the reference): the partial sums
    come as near to fp16's range as they can (six tiles of 128 rows a split), and
    the output is those rows' value, off by the weights' 2^-7 + 2^-11 and the
    partials' 2^-11."""
    T, k, sm = 40, 2048, 0.01                              # 3 splits a token
    s = Seqs(dsa, torch, [2100], [T])
    x = torch.full((s.rows, 576), 448.0, device="cuda")
    x[:, 512:] = 0.0
    at = torch.arange(s.rows, device="cuda")
    x[at // 128 % 6 > 0, 512] = 415.0                      # 2^5.987 times the first tile's weight, 2^2
    b = dsa.Batch.from_host([0, s.rows], range(s.rows), [0], s.rows)
    codes, scale = dsa.q8_cache(s.rows)
    dsa.dsa_kv_append_q8(x[:, :512], x[:, 512:], b, None, codes, scale, s.ws)
    q = torch.zeros(T, 64, 512, dtype=torch.bfloat16, device="cuda")
    qr = torch.zeros(T, 64, 64, dtype=torch.bfloat16, device="cuda")
    qr[:, :, 0] = 1.0
    idx = np.tile(np.arange(k, dtype=np.int32), (T, 1))
    out, _ = attend(dsa, torch, s, q, qr, codes, scale, idx, sm)
    assert ((out - 448.0).abs() <= 448.0 * (2.0 ** -7 + 2.0 ** -10)).all(), (float(out.min()), float(out.max()))
