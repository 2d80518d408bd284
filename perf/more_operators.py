"""Workloads of the dense attention over the latent cache, its sliding-window
form, and the norms in front of both: what a serving step runs in the layers
(and over the contexts) that select nothing, and before its projections.

Four operators, each in a plain form (elementary torch operations) and, where
`own` is true, as a program calls it from dsa_sparse_attention_score_gb300:

attn     softmax attention of every query head of a chunk of new tokens over
         all the latent rows its sequence has cached up to each token, in
         contiguous or paged caches; one token per sequence is decode
window   the same over the last `window` positions of each token and the first
         `sinks` positions of its sequence
norm     root-mean-square norm of rows, with the residual's addition
norm_q8  the same with e4m3 codes and one scale per group of values as output

A latent row is 576 bf16 values (512 latent | 64 rotary tail), or 512 without
a tail.  A token at position -1 is padding: it sees nothing, its output is 0 and
its log-sum-exp -infinity.
"""
import math

import numpy as np
import torch

own = False

LAT, TAIL = 512, 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TOP, LEAST = 448.0, 2.0 ** -40      # the largest e4m3 value; the least scale
EPS = 1e-6


# ------------------------------------------------------------------- cases

def _attn(name, seqs, per, lo, hi, heads, tail, page, window=0, sinks=0, padded=False):
    """The last `per` tokens of each of seqs sequences of lo..hi positions; the
    first token is padding when `padded`.  window 0: all positions."""
    c = dict(op="window" if window else "attn", seqs=seqs, per=per, lo=lo, hi=hi, heads=heads, tail=tail, page=page,
             window=window, sinks=sinks, padded=padded)
    return dict(c, name=name) if name else c


def _norm(name, rows, dim, width, dtype, residual, group=0):
    """rows of `dim` values, the first of `width` stored ones; group 0: no codes."""
    c = dict(op="norm_q8" if group else "norm", rows=rows, dim=dim, width=width, dtype=dtype, residual=residual, group=group)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the next token of one short conversation
        _attn("attn one token", 1, 1, 300, 300, 16, True, 64),
        # batched decode: 8 sequences of 8192 positions
        _attn("attn decode", 8, 1, 8192, 8192, 64, True, 0),
        # ragged decode of a 128-head model, paged
        _attn("attn decode ragged", 32, 1, 4096, 65536, 128, True, 64),
        # a prefill chunk after 6144 cached positions
        _attn("attn prefill", 1, 2048, 8192, 8192, 64, True, 0),
        # chunks of several prompts together, rows without a tail, pages of 16, an odd number of heads
        _attn("attn chunks", 5, 257, 1000, 5003, 33, False, 16),
        # decode through a window of 4096 with 64 sinks, paged
        _attn("window decode", 32, 1, 4096, 65536, 64, True, 64, 4096, 64),
        # a prefill chunk of a sliding-window layer
        _attn("window prefill", 1, 2048, 8192, 8192, 64, True, 0, 1000, 4),
        # the residual stream of 8 decoding sequences
        _norm("norm decode", 8, 4096, 4096, "bf16", True),
        # the latents of a chunk, as the projection left them ([latent | tail] rows), before they are cached
        _norm("norm latent", 4093, LAT, LAT + TAIL, "bf16", False),
        # the residual stream of a long prompt
        _norm("norm prefill", 16384, 7168, 7168, "bf16", True),
        # 8-bit inputs of the next projection: decode and a prompt
        _norm("norm q8 decode", 32, 7168, 7168, "bf16", True, 128),
        _norm("norm q8 prefill", 8191, 4096, 4096, "f16", True, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "window", "window", "norm", "norm_q8"])
    if op in ("norm", "norm_q8"):
        group = 0 if op == "norm" else rng.choice([32, 64, 128])
        dim = rng.choice([128 * _log(rng, 1, 80), 512, 1536]) if group else rng.choice([_log(rng, 1, 10000), 512, 4096])
        dtype = rng.choice(["bf16", "f16", "f32"])
        rows = _log(rng, 1, min(60000, (16384 * 7168 // 2) // dim))
        return _norm(None, rows, dim, dim + rng.choice([0, 0, 64, 7]), dtype, rng.random() < 0.6, group)
    heads = rng.choice([1, 5, 8, 16, 33, 64, 128])
    seqs = _log(rng, 1, 40)
    per = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, min(2048, 131072 // heads) // seqs))
    most = min(30000 if per > 1 else 60000, (2048 * 64 * 7000) // (seqs * per * heads), (2 << 20) // seqs)
    lo = per + _log(rng, 1, max(1, most - per)) // 2
    hi = lo + _log(rng, 1, max(1, most - lo))
    window = _log(rng, 1, 4096) if op == "window" else 0
    return _attn(None, seqs, per, lo, hi, heads, rng.random() < 0.75, rng.choice([0, 16, 64, 128]), window,
                 rng.choice([0, 1, 4, 64, 200]) if window else 0, rng.random() < 0.25)


def _lens(c):
    n = c["seqs"]
    return [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, n - 1) for b in range(n)]


def _visible(c, pos):
    """How many positions a token at pos sees (an array of positions)."""
    if not c["window"]:
        return pos + 1
    first = np.maximum(0, pos - c["window"] + 1)
    return pos + 1 - first + np.minimum(c["sinks"], first)


def work(c):
    if c["op"] in ("norm", "norm_q8"):
        n, e = c["rows"] * c["dim"], 4 if c["dtype"] == "f32" else 2
        out = n + 4 * c["rows"] * (c["dim"] // c["group"]) if c["group"] else n * e
        return {"bytes": n * e * (3 if c["residual"] else 1) + out + c["dim"] * e, "flops": 4 * n}
    wide = LAT + (TAIL if c["tail"] else 0)
    tokens, h = c["seqs"] * c["per"], c["heads"]
    pairs = rows = 0
    for n in _lens(c):
        pos = np.arange(n - c["per"], n)
        pairs += int(_visible(c, pos).sum())
        first = max(0, n - c["per"] - c["window"] + 1) if c["window"] else 0
        rows += n - first + min(c["sinks"], first)
    return {"bytes": rows * wide * 2 + tokens * h * (2 * wide + 2 * LAT + 4) + 4 * tokens, "flops": 2 * pairs * h * (wide + LAT)}


# ------------------------------------------------------------------ inputs

def _layout(c, g):
    """Where the sequences' positions lie: kv_off, block table and the row count."""
    lens = _lens(c)
    if not c["page"]:
        off = np.cumsum([0] + [n + 3 for n in lens])
        return torch.tensor(off[:-1], dtype=torch.int64, device="cuda"), None, int(off[-1])
    bs = c["page"]
    blocks = torch.tensor([-(-n // bs) for n in lens], device="cuda")
    total = int(blocks.sum()) + 2
    at = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(blocks, 0) - blocks
    col = torch.arange(int(blocks.max()), device="cuda")
    table = torch.where(col < blocks[:, None], at[(first[:, None] + col).clamp(max=total - 1)], -1)
    return torch.zeros(c["seqs"], dtype=torch.int64, device="cuda"), table.contiguous(), total * bs


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    s = {"case": c}
    if c["op"] in ("norm", "norm_q8"):
        dt, n, d = DTYPES[c["dtype"]], c["rows"], c["dim"]
        size = torch.exp2(normal(n, 1))            # tokens differ in size
        s["x"] = (normal(n, c["width"]) * size).to(dt)[:, :d]
        s["residual"] = (normal(n, d) * (4.0 * size)).to(dt) if c["residual"] else None
        s["sum"] = torch.empty(n, d, dtype=dt, device="cuda") if c["residual"] else None
        s["weight"] = (1.0 + 0.2 * normal(d)).to(dt)
        if c["group"]:
            s["codes"] = torch.empty(n, d, dtype=torch.uint8, device="cuda")
            s["scale"] = torch.empty(n, d // c["group"], device="cuda")
        else:
            s["out"] = torch.empty(n, d, dtype=dt, device="cuda")
        return s

    lens, per = _lens(c), c["per"]
    tokens, h = c["seqs"] * per, c["heads"]
    wide = LAT + (TAIL if c["tail"] else 0)
    s["off"], s["table"], rows = _layout(c, g)
    pos = (torch.tensor(lens, device="cuda")[:, None] - per + torch.arange(per, device="cuda")).flatten().to(torch.int32)
    if c["padded"]:
        pos[0] = -1
    s["pos"], s["rows"], s["max_kv"] = pos, rows, max(lens)
    s["cu_q"] = torch.arange(0, tokens + 1, per, dtype=torch.int32, device="cuda")
    s["kv"] = normal(rows, wide, dtype=torch.bfloat16)
    s["q_lat"] = normal(tokens, h, LAT, dtype=torch.bfloat16)
    s["q_rope"] = normal(tokens, h, TAIL, dtype=torch.bfloat16) if c["tail"] else None
    s["sm"] = 1.0 / math.sqrt(192.0 if c["tail"] else 256.0)
    s["out"] = torch.empty(tokens, h, LAT, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(tokens, h, device="cuda")
    if own:  # the handles such a program keeps
        import dsa_sparse_attention_score_gb300 as dsa
        s["batch"] = dsa.Batch(s["cu_q"], s["pos"], s["off"], per, s["max_kv"], rows)
        s["ws"] = dsa.workspace(dsa.DSA_OP_MLA_ATTN, s["batch"], H=h)
    return s


# -------------------------------------------------------------- plain forms

def _attend(s, c):
    B, per, h, M = c["seqs"], c["per"], c["heads"], s["max_kv"]
    at = torch.arange(M, device="cuda")
    pos = s["pos"].view(B, per, 1).long()
    seen = at <= pos
    if c["window"]:
        seen = seen & ((at > pos - c["window"]) | (at < c["sinks"]))
    used = seen.any(1)                                       # [B, M]
    if s["table"] is None:
        row = s["off"][:, None] + at
    else:
        row = s["table"].long().repeat_interleave(c["page"], 1)[:, :M] * c["page"] + at % c["page"]
    kv = s["kv"][torch.where(used, row, 0)].float()          # [B, M, wide]
    q = s["q_lat"] if s["q_rope"] is None else torch.cat((s["q_lat"], s["q_rope"]), -1)
    z = torch.matmul(q.float().view(B, per * h, -1), kv.transpose(1, 2)).mul_(s["sm"]).view(B, per, h, M)
    z.masked_fill_(~seen[:, :, None], -math.inf)
    top = z.amax(3, keepdim=True).clamp_(min=-1e30)
    p = z.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p.view(B, per * h, M), kv[..., :LAT]).view(B, per, h, LAT) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(out.view(-1, h, LAT))
    s["lse"].copy_((top + torch.log(total)).view(-1, h))     # log 0 = -infinity
    return {"out": s["out"], "lse": s["lse"]}


def _normalise(s, c):
    dt = s["x"].dtype
    x = s["x"].float()
    if s["residual"] is not None:
        s["sum"].copy_((x + s["residual"].float()).to(dt))
        x = s["sum"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    if not c["group"]:
        s["out"].copy_(y.to(dt))
        return {"out": s["out"], "sum": s["sum"]} if c["residual"] else s["out"]
    y = y.view(c["rows"], -1, c["group"])
    scale = (y.abs().amax(2, keepdim=True) / TOP).clamp(min=LEAST)
    s["codes"].copy_((y / scale).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8).view(c["rows"], -1))
    s["scale"].copy_(scale[..., 0])
    return _coded(s, c)


def _coded(s, c):
    """The codes as the values they stand for; the buffers themselves."""
    out = {"codes": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"]}
    return dict(out, sum=s["sum"]) if c["residual"] else out


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return _normalise(s, c) if c["op"] in ("norm", "norm_q8") else _attend(s, c)


def _run_own(s, c):
    import dsa_sparse_attention_score_gb300 as dsa
    if c["op"] == "norm":
        dsa.dsa_rms_norm(s["x"], s["residual"], s["sum"], s["weight"], EPS, s["out"])
        return {"out": s["out"], "sum": s["sum"]} if c["residual"] else s["out"]
    if c["op"] == "norm_q8":
        dsa.dsa_rms_norm_q8(s["x"], s["residual"], s["sum"], s["weight"], EPS, s["codes"], s["scale"])
        return _coded(s, c)
    page = (s["table"], c["page"]) if c["page"] else (None, 0)
    if c["op"] == "attn":
        dsa.dsa_mla_attn(s["q_lat"], s["q_rope"], s["kv"], s["batch"], s["sm"], s["out"], s["lse"], s["ws"], *page)
    else:
        dsa.dsa_mla_attn_window(s["q_lat"], s["q_rope"], s["kv"], s["batch"], c["window"], c["sinks"], None, s["sm"],
                                s["out"], s["lse"], s["ws"], *page)
    return {"out": s["out"], "lse": s["lse"]}


# -------------------------------------------------------------------- exact

def _nearest_e4m3(v):
    """The e4m3 value next to each |v| <= 448 (ties to the even one), in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 4, min=-9))
    return torch.clamp(torch.round(v / step) * step, -TOP, TOP)


def _exact_norm(s, c):
    x = s["x"].double()
    if c["residual"]:
        # the sum as it is stored: the row's own type
        kept = (x + s["residual"].double()).to(s["x"].dtype).double()
        x = kept
    y = x / torch.sqrt(torch.mean(x * x, 1, keepdim=True) + EPS) * s["weight"].double()
    if not c["group"]:
        return {"out": y, "sum": kept} if c["residual"] else y
    groups = y.unflatten(1, (c["dim"] // c["group"], c["group"]))
    step = torch.maximum(groups.abs().max(2).values / TOP, torch.tensor(LEAST, dtype=torch.float64, device="cuda"))
    out = {"codes": _nearest_e4m3(groups / step[..., None]).flatten(1), "scale": step}
    return dict(out, sum=kept) if c["residual"] else out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] in ("norm", "norm_q8"):
        return _exact_norm(s, c)
    outs, lses = [], []
    per, h = c["per"], c["heads"]
    for b, n in enumerate(_lens(c)):
        at = torch.arange(n, device="cuda")
        if c["page"]:
            rows = s["table"][b][torch.div(at, c["page"], rounding_mode="floor")].long() * c["page"] + torch.remainder(at, c["page"])
        else:
            rows = s["off"][b] + at
        many = max(1, (1 << 28) // (n * h))
        # the rows that nobody of the chunk sees are left out
        first = max(0, n - per - c["window"] + 1) if c["window"] else 0
        kept = torch.cat((at[:min(c["sinks"], first)], at[first:]))
        kv = s["kv"][rows[kept]].double()
        for t0 in range(b * per, (b + 1) * per, many):
            t = slice(t0, min(t0 + many, (b + 1) * per))
            z = torch.einsum("thd,kd->thk", s["q_lat"][t].double(), kv[:, :LAT])
            if c["tail"]:
                z = z + torch.einsum("thd,kd->thk", s["q_rope"][t].double(), kv[:, LAT:])
            p = s["pos"][t].long()[:, None]
            out_of_sight = kept > p
            if c["window"]:
                out_of_sight |= (kept <= p - c["window"]) & (kept >= c["sinks"])
            z = (z * s["sm"]).masked_fill_(out_of_sight[:, None], -math.inf)
            lses.append(torch.logsumexp(z, 2))
            w = torch.exp(z - torch.where(torch.isfinite(lses[-1]), lses[-1], 0.0)[..., None])
            outs.append(torch.einsum("thk,kd->thd", w, kv[:, :LAT]))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
