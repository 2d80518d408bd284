"""Float64 definitions of the rotary positions, the 8-bit latent row and the
attention over it, for the tests (numpy; nothing shared with the library).

Error bounds used by the tests, all from the number of roundings:
  half step of a type        eps / 2 of the value (bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4)
  turned pair (a, b)         the angle's fraction of a turn is rounded once to 32 bits
                             (2 pi 2^-25 < 2^-22 radians), sine and cosine are good to
                             2 units of 2^-24, the factor and the products round 3 times:
                             together under 2^-20 scale (|a| + |b|), then the half step
"""
import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def e4m3_round(v):
    """The e4m3 value nearest to v (ties to even), saturating at 448."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(v)
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def e4m3_decode(codes):
    b = np.asarray(codes).astype(np.int64)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e > 0, (1 + m / 8) * np.exp2(e - 7.0), m * 2.0 ** -9)
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def exponent(top):
    """Least E in [-40, 119] with top <= 448 2^E."""
    E = np.full(np.shape(top), -40)
    for n in range(-40, 119):
        E = np.where(top > 448.0 * 2.0 ** n, n + 1, E)
    return E


def rotate(x, pos, freq, scale, interleaved, inverse=False):
    """x [T, ..., 2n] in float64 turned by pos * freq; and scale (|a| + |b|) per value."""
    x = np.asarray(x, np.float64)
    n = len(freq)
    ang = np.multiply.outer(np.asarray(pos, np.float64), freq).reshape((x.shape[0],) + (1,) * (x.ndim - 2) + (n,))
    ang = -ang if inverse else ang
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :n], x[..., n:])
    ya, yb = scale * (a * np.cos(ang) - b * np.sin(ang)), scale * (a * np.sin(ang) + b * np.cos(ang))
    size = abs(scale) * (np.abs(a) + np.abs(b))
    y, s = np.empty_like(x), np.empty_like(x)
    if interleaved:
        y[..., 0::2], y[..., 1::2], s[..., 0::2], s[..., 1::2] = ya, yb, size, size
    else:
        y[..., :n], y[..., n:], s[..., :n], s[..., n:] = ya, yb, size, size
    return y, s


def quantise(lat, tail=None):
    """(values [n, 640 or 512], scale [n]) the codes of float64 rows stand for."""
    top = np.abs(lat).max(1)
    if tail is not None:
        top = np.maximum(top, np.abs(tail).max(1))
    s = np.exp2(exponent(top).astype(np.float64))[:, None]
    parts = [e4m3_round(lat / s)]
    if tail is not None:
        hi = e4m3_round(tail / s)
        parts += [hi, e4m3_round(tail / s - hi)]
    return np.concatenate(parts, 1), s[:, 0]


def encode(values):
    """Codes of e4m3 values."""
    table = e4m3_decode(np.arange(127))                     # 0 .. 448, ascending
    v = np.abs(values)
    at = np.searchsorted(table, v)
    assert np.array_equal(table[at], v)
    return (at + np.where(np.signbit(values), 128, 0)).astype(np.uint8)


def decode_rows(codes, scale):
    """(latent, tail or None) in float64."""
    v = e4m3_decode(codes) * np.asarray(scale, np.float64)[..., None]
    return (v[..., :512], v[..., 512:576] + v[..., 576:]) if codes.shape[-1] == 640 else (v, None)


def attention(q_lat, q_rope, codes, scale, rows, sm):
    """One token: q [H, .], rows the cache rows of its valid selections.
    Returns out [H, 512], lse [H] and the error bounds of both for the 8-bit
    product scheme:
      q is two e4m3 pieces under a power of two with 448 2^e >= its head's
      largest value: off by at most max(2^-8 |q|, 2^-10 2^e), 2^e <= top / 224
      (and 2^e >= 2^-40);
      sums of 640 products in 32 bits: under 2^-18 of the sum of magnitudes;
      a weight w_j 2^E_j is rounded to fp16 (2^-11) and split into an e4m3
      piece (off by 2^-4 of it, or 2^-10) and an e5m2 remainder (2^-3 of the
      remainder, or 2^-17), in units where the largest lies in [2^2, 2^8]: off
      by at most 2^-7 + 2^-11 of itself or 2^-13 + 2^-17, under 2^-14.9 of the
      largest;
      partial outputs of splits are bf16 (half step of at most sum w |c|);
      exponentials and their sums in 32 bits: 2^-18."""
    H = q_lat.shape[0]
    lat, tail = decode_rows(codes[rows], scale[rows])
    q, kv = (q_lat, lat) if tail is None else (np.concatenate([q_lat, q_rope], 1), np.concatenate([lat, tail], 1))
    if len(rows) == 0:
        return np.zeros((H, 512)), np.full(H, -np.inf), np.zeros((H, 512)), np.zeros(H)
    z = sm * q @ kv.T
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    L = p.sum(1, keepdims=True)
    w = p / L
    out, lse = w @ lat, (m + np.log(L))[:, 0]
    # q's pieces, then the sums
    step = np.maximum(np.abs(q).max(1, keepdims=True) / 224.0, 2.0 ** -40)
    dq = np.where(np.abs(q) > 0, np.minimum(np.maximum(2.0 ** -8 * np.abs(q), 2.0 ** -10 * step), np.abs(q)), 0.0)
    exact = np.abs(q) >= 2.0 ** -2 * step * 2               # eight bits fit the two pieces
    dq = np.where(exact, 0.0, dq)
    dz = abs(sm) * (dq @ np.abs(kv).T + 2.0 ** -18 * np.abs(q) @ np.abs(kv).T)
    dz = dz.max(1, keepdims=True)
    A = w @ np.abs(lat)
    s = np.asarray(scale, np.float64)[rows]
    top = (w * s).max(1, keepdims=True)
    code_sum = np.abs(e4m3_decode(codes[rows])[:, :512]).sum(0)[None, :]
    d_out = (2.0 ** -7 + 2.0 ** -11 + 2.0 ** -8 + 2.0 ** -18 + 2 * dz) * A + 2.0 ** -14.9 * top * code_sum
    d_lse = dz[:, 0] + 2.0 ** -18 * (1 + np.abs(lse))
    return out, lse, d_out, d_lse
