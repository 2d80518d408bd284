"""Windows and numbers of first positions that 32 bits do not hold."""
import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402
from _mla_ref import Case, check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,n_sink", [(2 ** 32 + 5, 0), (2 ** 40, 3), (7, 2 ** 32 + 2), (2 ** 31, 2 ** 63)])
def test_beyond_32_bits_is_everything(window, n_sink):
    c = Case([0, 3], [200, 50, 201], 16, lens=[202]).cuda()
    out, lse = c.run(dsa, window=window, n_sink=n_sink)
    check(out, lse, c.reference())


@pytest.mark.parametrize("window,n_sink", [(-2 ** 32 + 5, 0), (7, -2 ** 32 + 2), (0, 0), (7, -1)])
def test_below_is_refused(window, n_sink):
    c = Case([0, 3], [200, 50, 201], 16, lens=[202]).cuda()
    with pytest.raises(dsa.DsaError):
        c.run(dsa, window=window, n_sink=n_sink)
