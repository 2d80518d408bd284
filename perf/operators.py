"""Workloads of the 8-bit latent cache and its rotary positions: what a
serving step runs around the sparse attention.

Four operators, each in a plain form (elementary torch operations) and, where
`own` is true, as a program calls it from dsa_sparse_attention_score_gb300:

rope    rotary positions of head rows: interleaved or half layout, the whole
        head or a part of it, plain or context-scaled frequencies, forward or
        inverse (the gradient)
append  one latent row per new token, its tail rotated at the token's
        position, into the cache: 8-bit rows (e4m3 codes and one power-of-two
        scale per row; the tail as two codes, value and remainder) or bf16 rows
read    rows of the 8-bit cache back as bf16
attn    softmax attention of every query head over selected rows of the
        8-bit cache

The cache of a token is 640 codes (512 latent | 64 tail | 64 tail remainder;
512 without a tail) and one float32 scale 2^E, E the least integer in
[-40, 119] with max |x| <= 448 * 2^E.
"""
import math

import numpy as np
import torch

own = False

LAT, TAIL = 512, 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E_MIN, E_MAX, TOP = -40, 119, 448.0


# ------------------------------------------------------------------- cases

def _rope(name, tokens, heads, width, off, dim, rot, layout, dtype, scaling, far, inverse=False):
    """tokens rows of `heads` heads; each head is the slice [off, off + dim) of
    `width` stored values, its first `rot` values rotated; positions up to far."""
    c = dict(op="rope", tokens=tokens, heads=heads, width=width, off=off, dim=dim, rot=rot, layout=layout,
             dtype=dtype, scaling=scaling, far=far, inverse=inverse)
    return dict(c, name=name) if name else c


def _append(name, cache, seqs, per, lo, hi, tail, layout, dtype, scaling, page):
    """`per` new tokens of each of seqs sequences of lo..hi positions; cache "q8" or "bf16"."""
    c = dict(op="append", cache=cache, seqs=seqs, per=per, lo=lo, hi=hi, tail=tail, layout=layout, dtype=dtype,
             scaling=scaling, page=page)
    return dict(c, name=name) if name else c


def _read(name, seqs, per, lo, hi, tail, page):
    """The last `per` rows of each of seqs sequences of lo..hi positions."""
    c = dict(op="read", seqs=seqs, per=per, lo=lo, hi=hi, tail=tail, page=page)
    return dict(c, name=name) if name else c


def _attn(name, seqs, per, lo, hi, heads, k, tail, page, empty=False):
    """`per` query tokens at the end of each of seqs sequences of lo..hi positions."""
    c = dict(op="attn", seqs=seqs, per=per, lo=lo, hi=hi, heads=heads, k=k, tail=tail, page=page, empty=empty)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the tails of 8 decode queries, taken where the up-projection left them ([nope | tail] per head)
        _rope("rope decode q", 8, 64, 192, 128, 64, 64, "interleaved", "bf16", "none", 8192),
        # the tails of a prefill chunk of a 128-head model beyond its trained length
        _rope("rope prefill q long", 4096, 128, 192, 128, 64, 64, "interleaved", "bf16", "yarn", 131072),
        # indexer queries of a prefill chunk: the first half of each 128-wide head turns, half layout
        _rope("rope indexer q", 4093, 64, 128, 0, 128, 64, "half", "f16", "none", 65536),
        # the gradient of the rotated tails of a fine-tuning sequence
        _rope("rope gradient", 2047, 64, 64, 0, 64, 64, "interleaved", "f32", "linear", 4096, True),
        # one new latent row for each of 32 decoding sequences
        _append("append decode", "q8", 32, 1, 500, 4000, True, "interleaved", "bf16", "none", 64),
        # a long prompt's rows at once
        _append("append prefill", "q8", 1, 16384, 16384, 16384, True, "interleaved", "bf16", "yarn", 0),
        # one cached prompt handed to a bf16 consumer
        _read("read prompt", 1, 2048, 2048, 2048, True, 64),
        # the contexts of a ragged batch, paged
        _read("read contexts", 32, 3999, 4000, 8100, True, 64),
        # batched decode: 8 sequences of 8192 positions
        _attn("attn decode", 8, 1, 8192, 8192, 64, 2048, True, 0),
        # ragged decode: 32 sequences of 4k..64k positions, paged
        _attn("attn decode ragged", 32, 1, 4096, 65536, 64, 2048, True, 64),
        # decode of rows without a tail, pool-expanded selections of 2051
        _attn("attn decode no tail", 8, 1, 4000, 8191, 64, 2051, False, 0),
        # a prefill chunk after 4096 cached positions
        _attn("attn prefill", 1, 2048, 6144, 6144, 64, 2048, True, 0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attn", "attn"])
    scaling = rng.choice(["none", "linear", "yarn"])
    layout = rng.choice(["interleaved", "half"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "rope":
        heads = rng.choice([1, 5, 8, 16, 32, 64, 128])
        dim = rng.choice([64, 96, 128, 192])
        rot = rng.choice([32, 64, dim])
        off = rng.choice([0, 64])
        return _rope(None, _log(rng, 1, 4096 * 32 // max(32, heads)), heads, off + dim + rng.choice([0, 8, 64]), off, dim, rot, layout,
                     dtype, scaling, _log(rng, 4096, 1 << 20), rng.random() < 0.3)
    seqs = _log(rng, 1, 48)
    tail = rng.random() < 0.75
    page = rng.choice([0, 64, 128])
    if op == "append":
        per = rng.choice([1, _log(rng, 1, max(1, 12000 // seqs))])
        lo = per + _log(rng, 1, 2000)
        return _append(None, rng.choice(["q8", "q8", "bf16"]), seqs, per, lo, lo + _log(rng, 1, 2000), tail, layout, dtype,
                       scaling, page)
    if op == "read":
        per = _log(rng, 1, max(1, 60000 // seqs))
        return _read(None, seqs, per, per, per + _log(rng, 1, 4000), tail, page)
    heads = rng.choice([8, 16, 33, 64, 128])
    per = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, min(2048, 120000 // heads) // seqs))
    lo = per + _log(rng, 1, 8000)
    return _attn(None, seqs, per, lo, lo + _log(rng, 1, 30000 if per == 1 else 4000), heads, _log(rng, 1, 2048), tail, page,
                 rng.random() < 0.3)


def _lens(c):
    n = c["seqs"]
    return [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, n - 1) for b in range(n)]


def work(c):
    if c["op"] == "rope":
        n, e = c["tokens"] * c["heads"], 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2 * n * c["dim"] * e + 4 * c["tokens"], "flops": 3 * n * c["rot"]}
    row = (LAT + 2 * TAIL if c["tail"] else LAT) + 4
    wide = LAT + (TAIL if c["tail"] else 0)
    tokens = c["seqs"] * c["per"]
    if c["op"] == "append":
        out = row if c["cache"] == "q8" else 2 * wide
        return {"bytes": tokens * (wide * (4 if c["dtype"] == "f32" else 2) + out + 4), "flops": 4 * tokens * wide}
    if c["op"] == "read":
        return {"bytes": tokens * (row + 2 * wide + 4), "flops": tokens * wide}
    lens = _lens(c)
    seen = [min(c["k"], n - c["per"] + i + 1) for n in lens for i in range(c["per"])]
    rows = sum(min(n, sum(min(c["k"], n - c["per"] + i + 1) for i in range(c["per"]))) for n in lens)
    h = c["heads"]
    return {"bytes": rows * row + tokens * (h * (2 * wide + 2 * LAT + 4) + 4 * c["k"]),
            "flops": 2 * sum(seen) * h * (wide + LAT)}


# ------------------------------------------------------------------ inputs

def _frequencies(rot, scaling, base=10000.0, factor=8.0, trained=16384, fast=32.0, slow=1.0):
    """Turns per position of each pair, in radians, and the factor on the values."""
    j = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * j / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        at = lambda beta: rot * math.log(trained / (beta * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(0, math.floor(at(fast))), min(rot - 1, math.ceil(at(slow)))
        ramp = np.clip((j - low) / max(high - low, 1e-3), 0.0, 1.0)
        return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _layout(c, g):
    """Where the sequences' positions lie: kv_off, block table and the row count."""
    lens = _lens(c)
    if not c["page"]:
        off = np.cumsum([0] + [n + 3 for n in lens])
        return torch.tensor(off[:-1], dtype=torch.int64, device="cuda"), None, int(off[-1])
    bs = c["page"]
    blocks = [-(-n // bs) for n in lens]
    total = sum(blocks) + 2
    at = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["seqs"], max(blocks)), -1, dtype=torch.int32, device="cuda")
    first = np.cumsum([0] + blocks)
    for b, n in enumerate(blocks):
        table[b, :n] = at[int(first[b]):int(first[b]) + n]
    return None, table, total * bs


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"] in ("rope", "append"):
        f, scale = _frequencies(c["rot"] if c["op"] == "rope" else TAIL, c["scaling"])
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["rope_scale"] = scale
    if c["op"] == "rope":
        x = normal(c["tokens"], c["heads"], c["width"]).to(DTYPES[c["dtype"]])
        s["x"] = x[:, :, c["off"]:c["off"] + c["dim"]]
        s["pos"] = torch.randint(0, c["far"], (c["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        s["out"] = torch.empty(c["tokens"], c["heads"], c["dim"], dtype=x.dtype, device="cuda")
        return s

    lens = _lens(c)
    tokens, per = c["seqs"] * c["per"], c["per"]
    wide = LAT + (TAIL if c["tail"] else 0)
    off, table, rows = _layout(c, g)
    pos = np.concatenate([np.arange(n - per, n) for n in lens])
    s["cu_q"] = torch.arange(0, tokens + 1, per, dtype=torch.int32, device="cuda")
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    s["off"] = off if off is not None else torch.zeros(c["seqs"], dtype=torch.int64, device="cuda")
    s["table"], s["rows"] = table, rows
    s["max_q"], s["max_kv"] = per, max(lens)
    s["seq"] = torch.arange(c["seqs"], device="cuda").repeat_interleave(per)
    # latent rows of different sizes, as tokens have them
    size = torch.exp2(0.5 * normal(rows, 1))
    codes, scale = _quantise(normal(rows, LAT) * size, normal(rows, TAIL) * size if c["tail"] else None)
    s["codes"], s["scale"] = codes, scale
    if c["op"] == "append":
        x = (normal(tokens, wide) * torch.exp2(2.0 * normal(tokens, 1))).to(DTYPES[c["dtype"]])
        s["c_new"], s["r_new"] = x[:, :LAT], x[:, LAT:] if c["tail"] else None
        if c["cache"] == "bf16":
            s["kv"] = normal(rows, wide).to(torch.bfloat16)
            del s["codes"], s["scale"]
    elif c["op"] == "read":
        s["out"] = torch.empty(tokens, wide, dtype=torch.bfloat16, device="cuda")
    else:
        h, k = c["heads"], c["k"]
        s["q_lat"] = (0.5 * normal(tokens, h, LAT)).to(torch.bfloat16)
        s["q_rope"] = (0.5 * normal(tokens, h, TAIL)).to(torch.bfloat16) if c["tail"] else None
        s["sm"] = 1.0 / math.sqrt(192.0 if c["tail"] else 256.0)
        # a random subset of the visible positions, ascending, -1 behind it
        kk = min(k, max(lens))
        rank = torch.rand(tokens, max(lens), generator=g, device="cuda")
        rank.masked_fill_(torch.arange(max(lens), device="cuda")[None, :] > s["pos"][:, None], -1.0)
        best, at = rank.topk(kk, dim=1)
        at = torch.where(best >= 0, at, 1 << 40).sort(dim=1).values
        idx = torch.full((tokens, k), -1, dtype=torch.int32, device="cuda")
        idx[:, :kk] = torch.where(at < 1 << 40, at, -1).to(torch.int32)
        if c["empty"]:
            idx[0] = -1
        s["idx"] = idx
        s["out"] = torch.empty(tokens, h, LAT, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(tokens, h, device="cuda")
    if own:  # the handles such a program keeps
        import dsa_sparse_attention_score_gb300 as dsa
        b = s["batch"] = dsa.Batch(s["cu_q"], s["pos"], s["off"], s["max_q"], s["max_kv"], rows)
        s["ws"] = (dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, b, H=c["heads"], k=c["k"]) if c["op"] == "attn"
                   else dsa.workspace(dsa.DSA_OP_K_APPEND, b))
    return s


# -------------------------------------------------------------- plain forms

def _turn(x, pos, freq, scale, layout, inverse=False):
    """float32 rows x [T, ..., 2n] turned by pos * freq [n]."""
    n = freq.numel()
    angle = pos.double()[:, None] * freq
    cos, sin = (angle.cos() * scale).float(), (angle.sin() * (-scale if inverse else scale)).float()
    shape = [x.shape[0]] + [1] * (x.dim() - 2) + [n]
    cos, sin = cos.view(shape), sin.view(shape)
    a, b = (x[..., 0::2], x[..., 1::2]) if layout == "interleaved" else (x[..., :n], x[..., n:])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.stack((a, b), -1).flatten(-2) if layout == "interleaved" else torch.cat((a, b), -1)


def _quantise(lat, tail):
    """Codes (uint8) and scales of float32 rows."""
    top = lat.abs().amax(1)
    if tail is not None:
        top = torch.maximum(top, tail.abs().amax(1))
    m, e = torch.frexp(top)                               # top = m * 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(E_MIN, E_MAX)

    def two_to(n):
        return ((n.to(torch.int32) + 127) << 23).view(torch.float32)

    back = two_to(-e)[:, None]

    def code(v):
        return v.clamp(-TOP, TOP).to(torch.float8_e4m3fn)

    parts = [code(lat * back)]
    if tail is not None:
        r = tail * back
        hi = code(r)
        parts += [hi, code(r - hi.float())]
    codes = torch.cat([p.view(torch.uint8) for p in parts], 1)
    bad = ~torch.isfinite(top)
    scale = two_to(e)
    return torch.where(bad[:, None], torch.zeros_like(codes), codes), torch.where(bad, torch.full_like(scale, math.nan), scale)


def _rows(s, seq, pos):
    """Cache rows of positions pos of sequences seq (same shape)."""
    pos = pos.long()
    if s["table"] is None:
        return s["off"][seq] + pos
    bs = s["case"]["page"]
    return s["table"][seq, pos // bs].long() * bs + pos % bs


def _values(s, rows):
    """float32 latent rows (and tails) of the 8-bit cache."""
    v = s["codes"][rows].view(torch.float8_e4m3fn).float() * s["scale"][rows][..., None]
    if s["case"]["tail"]:
        v = torch.cat((v[..., :LAT], v[..., LAT:LAT + TAIL] + v[..., LAT + TAIL:]), -1)
    return v


def _cache_out(s):
    """The cache as the values its codes stand for; the buffers themselves."""
    if s["case"]["cache"] == "bf16":
        return {"kv": s["kv"]}
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"]}


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "rope":
        x = s["x"].float()
        y = _turn(x[..., :c["rot"]], s["pos"], s["freq"], s["rope_scale"], c["layout"], c["inverse"])
        s["out"].copy_(torch.cat((y, x[..., c["rot"]:]), -1))
        return s["out"]
    if c["op"] == "append":
        lat, tail = s["c_new"].float(), None
        if c["tail"]:
            tail = _turn(s["r_new"].float(), s["pos"], s["freq"], s["rope_scale"], c["layout"])
        rows = _rows(s, s["seq"], s["pos"])
        if c["cache"] == "bf16":
            s["kv"][rows] = (lat if tail is None else torch.cat((lat, tail), 1)).to(torch.bfloat16)
        else:
            s["codes"][rows], s["scale"][rows] = _quantise(lat, tail)
        return _cache_out(s)
    if c["op"] == "read":
        s["out"].copy_(_values(s, _rows(s, s["seq"], s["pos"])))
        return s["out"]
    idx = s["idx"]
    seen = idx >= 0
    kv = _values(s, _rows(s, s["seq"][:, None].expand_as(idx), idx.clamp(min=0)))
    q = s["q_lat"].float() if s["q_rope"] is None else torch.cat((s["q_lat"], s["q_rope"]), -1).float()
    z = torch.matmul(q, kv.transpose(1, 2)).mul_(s["sm"]).masked_fill_(~seen[:, None, :], -math.inf)
    top = z.amax(2, keepdim=True).clamp(min=-1e30)
    p = torch.exp(z - top)
    total = p.sum(2, keepdim=True)
    out = torch.matmul(p, kv[..., :LAT]) / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(out)
    s["lse"].copy_(torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))[..., 0])
    return {"out": s["out"], "lse": s["lse"]}


def _run_own(s, c):
    import dsa_sparse_attention_score_gb300 as dsa
    if c["op"] == "rope":
        rope = dsa.Rope(s["freq"], c["layout"] == "interleaved", s["rope_scale"])
        dsa.dsa_rope(s["x"], s["pos"], rope, s["out"], inverse=c["inverse"])
        return s["out"]
    page = (s["table"], c["page"]) if c["page"] else (None, 0)
    if c["op"] == "append":
        rope = dsa.Rope(s["freq"], c["layout"] == "interleaved", s["rope_scale"]) if c["tail"] else None
        if c["cache"] == "bf16":
            dsa.dsa_kv_append(s["c_new"], s["r_new"], s["batch"], rope, s["kv"], s["ws"], *page)
        else:
            dsa.dsa_kv_append_q8(s["c_new"], s["r_new"], s["batch"], rope, s["codes"], s["scale"], s["ws"], *page)
        return _cache_out(s)
    if c["op"] == "read":
        dsa.dsa_kv_read_q8(s["codes"], s["scale"], s["batch"], s["out"], s["ws"], *page)
        return s["out"]
    dsa.dsa_sparse_mla_attn_q8(s["q_lat"], s["q_rope"], s["codes"], s["scale"], s["batch"], s["idx"], s["sm"],
                               s["out"], s["lse"], s["ws"], *page)
    return {"out": s["out"], "lse": s["lse"]}


# -------------------------------------------------------------------- exact

def _exact_turn(x, s):
    """x [T, h, 2n] in 64 bits, as complex numbers times e^(i angle)."""
    c = s["case"]
    n = x.shape[-1] // 2
    z = torch.view_as_complex((x.unflatten(-1, (n, 2)) if c["layout"] == "interleaved" else x.unflatten(-1, (2, n)).transpose(-1, -2)).contiguous())
    angle = torch.outer(s["pos"].to(torch.float64), s["freq"])[:, None]
    turn = torch.polar(torch.full_like(angle, s["rope_scale"]), -angle if c.get("inverse") else angle)
    y = torch.view_as_real(z * turn)
    return (y if c["layout"] == "interleaved" else y.transpose(-1, -2)).flatten(-2)


def _nearest_e4m3(v):
    """The e4m3 value next to each |v| <= 464 (ties to the even one), in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 4, min=-9))
    return torch.clamp(torch.round(v / step) * step, -TOP, TOP)


def _decoded(codes):
    """e4m3 codes from their bits, in 64 bits."""
    b = codes.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).to(torch.float64)
    v = torch.where(e > 0, torch.ldexp(1.0 + m / 8.0, e - 7), torch.ldexp(m, torch.full_like(e, -9)))
    return torch.where(b >= 128, -v, v)


def _exact_rows(s, rows):
    v = _decoded(s["codes"][rows]) * s["scale"][rows].double().unsqueeze(-1)
    return (v[..., :LAT], v[..., LAT:LAT + TAIL] + v[..., LAT + TAIL:]) if s["case"]["tail"] else (v, None)


def _exact_place(s, b, pos):
    """The cache row of position pos of sequence b."""
    bs = s["case"]["page"]
    if not bs:
        return s["off"][b] + pos.long()
    return s["table"][b][torch.div(pos, bs, rounding_mode="floor").long()].long() * bs + torch.remainder(pos, bs).long()


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        x = s["x"].double()
        return torch.cat((_exact_turn(x[..., :c["rot"]], s), x[..., c["rot"]:]), -1)
    per = c["per"]
    if c["op"] == "append":
        new = s["c_new"].double()
        r = _exact_turn(s["r_new"].double()[:, None], s)[:, 0] if c["tail"] else None
        if c["cache"] == "bf16":
            kv = s["kv"].double()
        else:
            codes, scale = _decoded(s["codes"]), s["scale"].double()
            top = new.abs().max(1).values if r is None else torch.maximum(new.abs().max(1).values, r.abs().max(1).values)
            powers = torch.tensor([2.0 ** n for n in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device="cuda")
            step = powers[(top[:, None] > TOP * powers[:-1]).sum(1)][:, None]
            q = [_nearest_e4m3(new / step)]
            if r is not None:
                first = _nearest_e4m3(r / step)
                q += [first, _nearest_e4m3(r / step - first)]
        for b in range(c["seqs"]):
            t = slice(b * per, (b + 1) * per)
            at = _exact_place(s, b, s["pos"][t])
            if c["cache"] == "bf16":
                kv[at] = new[t] if r is None else torch.cat((new[t], r[t]), 1)
            else:
                codes[at], scale[at] = torch.cat([x[t] for x in q], 1), step[t, 0]
        return {"kv": kv} if c["cache"] == "bf16" else {"codes": codes, "scale": scale}
    if c["op"] == "read":
        got = []
        for b in range(c["seqs"]):
            lat, tail = _exact_rows(s, _exact_place(s, b, s["pos"][b * per:(b + 1) * per]))
            got.append(lat if tail is None else torch.cat((lat, tail), 1))
        return torch.cat(got)
    outs, lses = [], []
    many = max(1, (1 << 28) // (c["k"] * LAT))
    for b in range(c["seqs"]):
        for t0 in range(b * per, (b + 1) * per, many):
            t = slice(t0, min(t0 + many, (b + 1) * per))
            idx = s["idx"][t].long()
            lat, tail = _exact_rows(s, _exact_place(s, b, idx.clamp(min=0)))
            z = torch.einsum("thd,tkd->thk", s["q_lat"][t].double(), lat)
            if tail is not None:
                z = z + torch.einsum("thd,tkd->thk", s["q_rope"][t].double(), tail)
            z = torch.where((idx >= 0)[:, None], z * s["sm"], torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
            lses.append(torch.logsumexp(z, 2))
            w = torch.where(torch.isfinite(lses[-1])[..., None], torch.exp(z - lses[-1][..., None]), 0.0)
            outs.append(torch.einsum("thk,tkd->thd", w, lat))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
