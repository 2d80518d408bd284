"""dsa_rms_norm_q8's codes and scales bit for bit, where the norm's values are known
exactly: rows of +-1 with eps 0 have a root mean square of 1, so that the float32
weights (with the rows' signs) are the values that are coded.  scale = max(max |y| / 448,
2^-40) and y / scale are float32 quotients, the code their e4m3 rounding."""
import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402

pytestmark = pytest.mark.gpu


def ulps(v, k):
    """Float32 values k steps from v > 0."""
    return (v.view(torch.int32) + k).view(torch.float32)


def weights_on_borders(dim, group, seed, spread):
    """Groups whose quotients by the scale lie on the borders between two codes, and a step
    beside them."""
    g = torch.Generator().manual_seed(seed)
    n = dim // group
    top = (1 + torch.rand(n, 1, generator=g)) * torch.exp2(torch.randint(-spread, spread + 1, (n, 1), generator=g).float())
    codes = torch.arange(0, 0x7e, dtype=torch.uint8)          # 0 .. 416: the one behind each is a number too
    v = codes.view(torch.float8_e4m3fn).float()
    borders = (v + (codes + 1).view(torch.float8_e4m3fn).float()) / 2
    at = borders[torch.randint(0, len(borders), (n, group), generator=g)]
    w = ulps(at * (top / 448).clamp(min=2.0 ** -40), torch.randint(-1, 2, (n, group), generator=g, dtype=torch.int32))
    w[:, 3] = 0                                               # a code of 0 has its value's sign
    w[torch.arange(n), torch.randint(4, group, (n,), generator=g)] = top[:, 0]
    return w.reshape(dim)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim,group,spread", [(4096, 128, 30), (4096, 64, 0), (1536, 32, 80), (512, 512, 5), (16384, 16384, 3), (16, 16, 1),
                                              (7168, 128, 45)])
@pytest.mark.parametrize("shift", [0, 1])
def test_codes_are_those_of_the_quotients(dim, group, spread, dtype, shift):
    n = 200
    g = torch.Generator().manual_seed(dim + group)
    sign = (2 * torch.randint(0, 2, (n, dim), generator=g) - 1).float()
    w = weights_on_borders(dim, group, spread, spread)
    y = (sign * w).view(n, -1, group)
    scale = (y.abs().amax(2) / 448).clamp(min=2.0 ** -40)
    ref = (y / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(n, dim)
    wide = torch.empty(n, dim + shift, dtype=dtype, device="cuda")
    x = wide[:, shift:]
    x.copy_(sign)
    codes, got = torch.empty(n, dim, dtype=torch.uint8, device="cuda"), torch.empty(n, dim // group, device="cuda")
    dsa.dsa_rms_norm_q8(x, None, None, w.cuda(), 0.0, codes, got)
    assert torch.equal(got.cpu(), scale)
    assert torch.equal(codes.cpu(), ref), f"{int((codes.cpu() != ref).sum())} codes differ"
