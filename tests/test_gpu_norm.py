"""dsa_rms_norm and dsa_rms_norm_q8 against their definition in 64 bits.

The stored sum is the float32 sum rounded once: bit for bit.  In float32, h^2 sums
over chains of at most 32 terms and a tree of at most 10 + 32, all positive: 74
roundings of half a step (2^-24) at the most; its root halves that, division, eps,
root and the two products add 6: y is off by less than 48 * 2^-24 |y|, and the
output by its own rounding.  A scale is off by as much as the largest y (and a
division); a code by half a step of e4m3: 2^-4 of its value, or 2^-10 scales."""
import math

import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
Y = 48 * 2.0 ** -24


def rows(n, dim, dtype, seed, width=None, off=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, width or dim, generator=g) * size * torch.exp2(torch.randn(n, 1, generator=g))
    return x.to(dtype).cuda()[:, off:off + dim]


def definition(x, r, w, eps):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    d = h.double()
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    return h, y if w is None else y * w.double()


def check_out(out, y):
    err, tol = (out.double() - y).abs(), y.abs() * (Y + U[out.dtype] * (1 + Y))
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25                   # half the least step
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,dim", [(1, 1), (3, 7), (1, 128), (5, 512), (8, 4096), (2, 4095), (700, 576), (3, 7168), (1, 16384),
                                   (2, 16383), (1300, 1000), (9000, 40)])
def test_norm(n, dim, dtype):
    x, r = rows(n, dim, dtype, 1), rows(n, dim, dtype, 2, size=4.0)
    w = (1 + 0.2 * torch.randn(dim, device="cuda")).to(dtype)
    out, s = torch.empty_like(x), torch.empty_like(x)
    dsa.dsa_rms_norm(x, r, s, w, 1e-6, out)
    h, y = definition(x, r, w, 1e-6)
    assert torch.equal(s, h)
    check_out(out, y)
    dsa.dsa_rms_norm(x, None, None, None, 1e-5, out)
    check_out(out, definition(x, None, None, 1e-5)[1])


@pytest.mark.parametrize("dtype", TYPES)
def test_float32_weights_and_no_stored_sum(dtype):
    x, r = rows(6, 640, dtype, 3), rows(6, 640, dtype, 4)
    w = torch.randn(640, device="cuda")
    out = torch.empty_like(x)
    dsa.dsa_rms_norm(x, r, None, w, 1e-6, out)
    check_out(out, definition(x, r, w, 1e-6)[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width,off", [(576, 0), (576, 64), (583, 0), (600, 3)])
def test_column_slices(dtype, width, off):
    """Latents where a projection left them; the columns beside them stay."""
    big = rows(37, width, dtype, 5)
    x = big[:, off:off + 512]
    out_big = torch.full((37, width), 7.0, dtype=dtype, device="cuda")
    out = out_big[:, off:off + 512]
    w = torch.randn(512, device="cuda").to(dtype)
    dsa.dsa_rms_norm(x, None, None, w, 1e-6, out)
    check_out(out, definition(x, None, w, 1e-6)[1])
    assert (out_big[:, :off] == 7).all() and (out_big[:, off + 512:] == 7).all()


@pytest.mark.parametrize("dim", [512, 4096, 33])
def test_in_place(dim):
    x, r = rows(50, dim, torch.bfloat16, 6), rows(50, dim, torch.bfloat16, 7)
    h, y = definition(x, r, None, 1e-6)
    x1, r1 = x.clone(), r.clone()
    dsa.dsa_rms_norm(x1, r1, r1, None, 1e-6, x1)             # the usual step: both in place
    assert torch.equal(r1, h)
    check_out(x1, y)
    x1, r1 = x.clone(), r.clone()
    dsa.dsa_rms_norm(x1, r1, x1, None, 1e-6, r1)
    assert torch.equal(x1, h)
    check_out(r1, y)


def test_zero_rows_and_values_that_are_not_finite():
    x = rows(4, 256, torch.bfloat16, 8)
    x[1] = 0
    x[2, 5] = math.nan
    out = torch.empty_like(x)
    dsa.dsa_rms_norm(x, None, None, None, 1e-6, out)
    assert (out[1] == 0).all() and torch.isnan(out[2]).all()
    check_out(out[[0, 3]], definition(x[[0, 3]], None, None, 1e-6)[1])


def check_codes(codes, scale, y, group):
    n, dim = y.shape
    y = y.view(n, -1, group)
    top = y.abs().amax(2)
    ref = (top / 448).clamp(min=2.0 ** -40)
    assert ((scale.double() - ref).abs() <= ref * (Y + 2.0 ** -22)).all()
    v = codes.view(torch.float8_e4m3fn).double().view(n, -1, group)
    s = scale.double()[..., None]
    tol = y.abs() * (2.0 ** -4 + 2 * Y + 2.0 ** -21) + s * 2.0 ** -10
    assert ((v * s - y).abs() <= tol).all()
    full = top > 448 * 2.0 ** -39
    assert (v.abs().amax(2)[full] == 448).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,dim,group", [(1, 32, 32), (3, 128, 128), (32, 7168, 128), (5, 4096, 64), (700, 512, 512), (9, 1536, 32),
                                         (4, 16384, 16384), (6, 16, 16), (2, 10240, 128), (1500, 576, 576)])
def test_codes(n, dim, group, dtype):
    x, r = rows(n, dim, dtype, 9), rows(n, dim, dtype, 10, size=4.0)
    w = (1 + 0.2 * torch.randn(dim, device="cuda")).to(dtype)
    s = torch.empty_like(x)
    codes = torch.empty(n, dim, dtype=torch.uint8, device="cuda")
    scale = torch.empty(n, dim // group, device="cuda")
    dsa.dsa_rms_norm_q8(x, r, s, w, 1e-6, codes, scale)
    h, y = definition(x, r, w, 1e-6)
    assert torch.equal(s, h)
    check_codes(codes, scale, y, group)


def test_codes_of_slices_zeros_and_values_that_are_not_finite():
    big = rows(12, 583, torch.float16, 11)
    x = big[:, 3:515]
    x[2, :128] = 0
    x[4, 200] = math.inf
    w = torch.ones(512, dtype=torch.float16, device="cuda")
    w[300:310] = 0
    codes, scale = torch.empty(12, 512, dtype=torch.uint8, device="cuda"), torch.empty(12, 4, device="cuda")
    dsa.dsa_rms_norm_q8(x, None, None, w, 1e-6, codes, scale)
    assert (scale[2, 0] == 2.0 ** -40) and (codes[2, :128] == 0).all()
    # the root of infinity takes all finite values to 0 and the infinite one to NaN
    assert torch.isnan(scale[4]).tolist() == [False, True, False, False]
    assert (codes[4] & 0x7f == 0).all()
    keep = [i for i in range(12) if i != 4]
    check_codes(codes[keep], scale[keep], definition(x[keep], None, w, 1e-6)[1], 128)


def test_captured_and_replayed():
    x, r = rows(8, 4096, torch.bfloat16, 12), rows(8, 4096, torch.bfloat16, 13)
    out, s = torch.empty_like(x), torch.empty_like(x)
    dsa.dsa_rms_norm(x, r, s, None, 1e-6, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_rms_norm(x, r, s, None, 1e-6, out)
        dsa.dsa_rms_norm(out, s, s, None, 1e-6, out)
    x.copy_(rows(8, 4096, torch.bfloat16, 14))
    g.replay()
    torch.cuda.synchronize()
    h, y = definition(x, r, None, 1e-6)
    first = torch.empty_like(x)
    dsa.dsa_rms_norm(x, r, None, None, 1e-6, first)
    h2, y2 = definition(first, h, None, 1e-6)
    assert torch.equal(s, h2)
    check_out(out, y2)
