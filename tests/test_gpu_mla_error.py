"""How far attention over all visible rows is off in total (2-norm), against what its
roundings give.

A bf16 rounding is off by up to 2^-8 of a significand in [1, 2): of the value, with
significands spread as those of exponentials are (evenly in their logarithm), by
2^-8 / sqrt(3) * sqrt(3 / (8 ln 2)) = 0.425 * 2^-8 in the root of the mean square.  The
rounding errors of the probabilities are independent of each other and of the rows that
they multiply, whose entries are independent too: the outputs' squares sum to
sum p^2 |c|^2 and the errors' to (0.425 * 2^-8)^2 times that.  A float32 output is so
off by 0.425 * 2^-8 of its size; a bf16 one is rounded once more, by as much, and
may be joined from fp16 parts (an eighth of it): 0.425 * sqrt(2 + 1/64) = 0.603.  Over
hundreds of rows, each with tens of keys that count, the means hold to a few per cent; a
sixth is allowed on top."""
import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402
from _mla_ref import Case  # noqa: E402

pytestmark = pytest.mark.gpu
BOUND = {torch.bfloat16: 0.7 * 2.0 ** -8, torch.float32: 0.5 * 2.0 ** -8}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("window", [None, 200])
@pytest.mark.parametrize("lens,per", [([2000, 300, 90], [12, 20, 30]), ([4000] * 6, [1] * 6)])
def test_error_is_that_of_its_roundings(lens, per, window, block, dtype):
    cu, pos = [0], []
    for n, k in zip(lens, per):
        pos += range(n - k, n)
        cu.append(len(pos))
    kw = dict(window=window, n_sink=4) if window else {}
    c = Case(cu, pos, 64, block=block).cuda()
    got, lse = c.run(dsa, dtype=dtype, **kw)
    ref, ref_lse, _, tol_lse = c.reference(**kw)
    rel = float((got.double() - ref).norm() / ref.norm())
    assert rel <= BOUND[dtype], f"off by {rel * 256:.3f} * 2^-8"
    assert ((lse.double() - ref_lse).abs() <= tol_lse).all()
