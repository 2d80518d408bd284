"""Attention over all visible rows with bf16 outputs where some dims of the latents are
far smaller than those beside them: each is as close to its own value as the others,
also in rows that are joined from the parts of several clusters."""
import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402
from _mla_ref import Case, check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [1, 64])
@pytest.mark.parametrize("small", [2.0 ** -12, 2.0 ** -18, 2.0 ** -26])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 60, 2.0 ** -60])
def test_small_dims_beside_large_ones(size, small, H):
    c = Case([0, 1, 3], [9000, 700, 701], H, lens=[9001, 702])
    c.kv[:, :512:3] *= small
    c.kv[:, 96:128] = 0                                       # a whole unit of a part
    c.kv *= size
    c.q_lat *= 1 / size                                       # scores as without the sizes
    c.q_rope *= 1 / size
    c.cuda()
    out, lse = c.run(dsa, dtype=torch.bfloat16)
    assert dsa.dsa_read_device_status(c.ws) == 0
    check(out, lse, c.reference())
    assert (out[..., 96:128] == 0).all()
