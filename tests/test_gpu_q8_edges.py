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
