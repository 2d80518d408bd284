"""dsa_rms_norm over as many rows as a call can name."""
import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 4])
def test_the_last_of_2_to_the_31_rows(n):
    """Short rows share a CTA: the last CTA's threads count past 2^31 - 1."""
    x = torch.empty(n + 64, dtype=torch.float16, device="cuda")
    x.fill_(3.0)                                              # 4.3 GB, in place
    x[:n:4097] = -2.0
    dsa.dsa_rms_norm(x[:n, None], None, None, None, 0.0, x[:n, None])
    assert (x[n:] == 3).all()                                 # behind the last row
    assert (x[:n:4097] == -1).all()
    step = 1 << 28
    for a in range(0, n, step):                               # every other row gives 1
        part = x[a:min(a + step, n)]
        first = -a % 4097
        assert int((part == -1).sum()) == len(range(first, part.numel(), 4097))
        assert int((part == 1).sum()) == part.numel() - len(range(first, part.numel(), 4097))
