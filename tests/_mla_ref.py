"""Attention over all visible latent rows (or a window and the first ones) in
64 bits, from its definition, and how far the float32 / bf16 kernel may be off."""
from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}     # half a step, relative


def rows_of(positions, seq, kv_off, table, block):
    if table is None:
        return kv_off[seq].long() + positions
    return table[seq, positions // block].long() * block + positions % block


def attention(q_lat, q_rope, kv, cu_q, q_pos, kv_off, sm, table=None, block=0, window=None, n_sink=0, sink_pos0=None,
              rel_check=True):
    """out, lse (float64), and bounds on their errors: tol_out for a float32
    output (the rounding of another type comes on top), tol_lse.

    The kernel rounds each probability to bf16 (2^-8 of it) and sums in float32:
    out is off by at most (2^-8 + e) sum p |c| / sum p, e = twice what a score may
    be off (576 products and their sums at 2^-23 each, relative to sum |q c|)
    plus n sums of the value product at 2^-23 each; and lse by e + 2^-20.  For bf16
    outputs, rows that several clusters share are joined from parts o_k in fp16 with a
    unit for 32 dims, each off by at most 2^-11 |o_k| (2^-24 of the largest of the 32
    where that is more), together by 2^-11 sum |o_k| <= 2^-11 sum p |c| / sum p: an
    eighth of tol_out."""
    T, H, _ = q_lat.shape
    out = torch.zeros(T, H, 512, dtype=torch.float64, device=kv.device)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=kv.device)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    cu, pos = cu_q.tolist(), q_pos.tolist()
    for b in range(len(cu) - 1):
        for t in range(cu[b], cu[b + 1]):
            p = pos[t]
            if p < 0:
                continue
            lo = 0 if window is None else max(0, p - window + 1)
            s = set(range(lo, p + 1))
            if window is not None and n_sink:
                a = max(0, int(sink_pos0[b])) if sink_pos0 is not None else 0
                s |= set(range(a, min(a + n_sink, p + 1)))
            at = torch.tensor(sorted(s), device=kv.device)
            c = kv[rows_of(at, b, kv_off, table, block)].double()
            q = q_lat[t].double() if q_rope is None else torch.cat((q_lat[t], q_rope[t]), 1).double()
            z = sm * (q @ c.T)
            e = 576 * 2.0 ** -23 * (abs(sm) * (q.abs() @ c.abs().T)).amax(1)      # [H]
            w = torch.softmax(z, 1)
            out[t] = w @ c[:, :512]
            lse[t] = torch.logsumexp(z, 1)
            tol_o[t] = (w @ c[:, :512].abs()) * (2.0 ** -8 + 2 * e[:, None] + len(s) * 2.0 ** -23)
            tol_l[t] = e + 2.0 ** -20 * (1 + lse[t].abs())
    return out, lse, tol_o, tol_l


def check(got, got_lse, ref, name="mla"):
    out, lse, tol_o, tol_l = ref
    g = got.double()
    err = (g - out).abs()
    parts = 1.125 if got.dtype == torch.bfloat16 else 1.0
    tol = parts * tol_o + U[got.dtype] * (out.abs() + tol_o) + 1e-30
    assert torch.isfinite(g).all(), f"{name}: {int((~torch.isfinite(g)).sum())} outputs are not finite"
    assert (err <= tol).all(), f"{name}: out off by {float((err / tol).max()):.2f} of the bound"
    # The rounding errors of the probabilities are independent of the rows they
    # multiply: together they are at most as large, relative to the output, as
    # each (2^-8), and so are those of the parts (bf16 outputs) and of the output.
    norm = float(out.norm())
    if norm:
        rel = float((g - out).norm()) / norm
        assert rel <= parts * 2.0 ** -8 + U[got.dtype] + 2.0 ** -12, f"{name}: out off by {rel:.2e} (2-norm)"
    if got_lse is not None:
        gl = got_lse.double()
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(gl) & (gl < 0), empty), f"{name}: rows without a key"
        assert (g[empty] == 0).all()
        e = (gl - lse).abs()[~empty]
        assert (e <= tol_l[~empty]).all(), f"{name}: lse off by {float((e / tol_l[~empty]).max()):.2f} of the bound"


class Case:
    """A batch over a cache whose unused rows hold NaN."""

    def __init__(self, cu_q, q_pos, H, tail=True, block=0, seed=0, spare_rows=5, lens=None, q_size=1.0, kv_off=None, rows=None):
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.H, self.tail, self.block = len(cu_q) - 1, len(q_pos), H, tail, block
        width = 576 if tail else 512
        self.lens = lens or [max([p + 1 for p in q_pos[cu_q[b]:cu_q[b + 1]]] + [0]) for b in range(self.B)]
        self.max_kv = max(max(self.lens), 1)
        if block:
            need = [-(-n // block) for n in self.lens]
            total = sum(need) + 3
            ids = torch.randperm(total, generator=g)
            self.table = torch.full((self.B, max(max(need), -(-self.max_kv // block))), -1, dtype=torch.int32)
            k = 0
            for b, n in enumerate(need):
                self.table[b, :n] = ids[k:k + n].to(torch.int32)
                k += n
            self.rows = total * block
            self.kv_off = torch.zeros(self.B, dtype=torch.int64)
        else:
            self.table = None
            offs, at = [], 2
            for n in self.lens:
                offs.append(at)
                at += n + spare_rows
            self.kv_off = torch.tensor(offs if kv_off is None else kv_off, dtype=torch.int64)
            self.rows = at if rows is None else rows
        self.cu_q = torch.tensor(cu_q, dtype=torch.int32)
        self.q_pos = torch.tensor(q_pos, dtype=torch.int32)
        bf = torch.bfloat16
        self.q_lat = (q_size * torch.randn(self.T, H, 512, generator=g)).to(bf)
        self.q_rope = (q_size * torch.randn(self.T, H, 64, generator=g)).to(bf) if tail else None
        self.kv = torch.full((self.rows, width), math.nan, dtype=bf)
        for b, n in enumerate(self.lens):
            if n:
                r = rows_of(torch.arange(n), b, self.kv_off, self.table, block)
                self.kv[r] = torch.randn(n, width, generator=g).to(bf)
        self.sm = 1.0 / math.sqrt(192.0)

    def cuda(self):
        for k, v in list(vars(self).items()):
            if torch.is_tensor(v):
                setattr(self, k, v.cuda())
        return self

    def reference(self, **kw):
        return attention(self.q_lat, self.q_rope, self.kv, self.cu_q, self.q_pos, self.kv_off, self.sm, self.table,
                         self.block, **kw)

    def batch(self, dsa, max_q=None):
        cu = self.cu_q.tolist()
        most = max(b - a for a, b in zip(cu, cu[1:]))
        return dsa.Batch(self.cu_q, self.q_pos, self.kv_off, max_q or max(most, -(-self.T // self.B)), self.max_kv, self.rows)

    def run(self, dsa, window=None, n_sink=0, sink_pos0=None, dtype=torch.bfloat16, lse=True, ws=None, out=None):
        b = self.batch(dsa)
        if ws is None:
            ws = dsa.workspace(dsa.DSA_OP_MLA_ATTN, b, H=self.H)
        if out is None:
            out = torch.full((self.T, self.H, 512), 7.0, dtype=dtype, device="cuda")
        ls = torch.full((self.T, self.H), 7.0, device="cuda") if lse else None
        page = (self.table, self.block) if self.block else (None, 0)
        if window is None:
            dsa.dsa_mla_attn(self.q_lat, self.q_rope, self.kv, b, self.sm, out, ls, ws, *page)
        else:
            dsa.dsa_mla_attn_window(self.q_lat, self.q_rope, self.kv, b, window, n_sink, sink_pos0, self.sm, out, ls, ws, *page)
        self.ws = ws
        return out, ls
