"""Attention over all visible rows: NaN in a query stays in the outputs of its own row,
and is not taken for a row that sees nothing."""
import math

import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402
from _mla_ref import Case, check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [6, 129, 3000])
@pytest.mark.parametrize("window", [None, 70])
def test_queries_of_nan(window, n, dtype):
    """Items of one tile, of two, and such as several clusters share."""
    kw = dict(window=window, n_sink=2) if window else {}
    c = Case([0, 3, 4], [n - 3, n - 2, n - 1, 5], 24, lens=[n, 6]).cuda()
    ref = c.reference(**kw)
    bad = torch.zeros(4, 24, dtype=torch.bool, device="cuda")
    c.q_lat[1, 5, 17], c.q_lat[2, 23], c.q_rope[0, 0, 63], c.q_lat[3, 7, 511] = (math.nan,) * 4
    for t, h in ((1, 5), (2, 23), (0, 0), (3, 7)):
        bad[t, h] = True
    out, lse = c.run(dsa, dtype=dtype, **kw)
    assert dsa.dsa_read_device_status(c.ws) == 0
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    check(out[~bad], lse[~bad], tuple(x[~bad] for x in ref))


@pytest.mark.parametrize("n", [1, 500])
def test_rows_of_nan(n):
    """All that a token sees."""
    c = Case([0, 1, 2], [n - 1, 40], 16, lens=[n, 41]).cuda()
    ref = c.reference()
    off = int(c.kv_off[0])
    c.kv[off:off + n] = math.nan
    out, lse = c.run(dsa)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    check(out[1:], lse[1:], tuple(x[1:] for x in ref))
