"""Attention over all visible rows and through a window where tokens that are not in
order (out of bounds, or in an unmapped block) share their query rows' work with
tokens that are: those are as without them, whatever unseen rows hold."""
import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402
from _mla_ref import Case, check  # noqa: E402
from test_gpu_mla_gaps import ANY, hide  # noqa: E402

pytestmark = pytest.mark.gpu


def leave_row_0(c):
    """Nothing in the cache's first block."""
    used, u = set(c.table.flatten().tolist()), 0
    while u in used or u == 0:
        u += 1
    c.kv[u * c.block:(u + 1) * c.block] = c.kv[:c.block].clone()
    c.table[c.table == 0] = u
    return c


def run_beside(c, bad, window=None, n_sink=0, status=None, only=None):
    """Runs with the tokens `bad` out of order: empty and flagged, the others in bounds."""
    kw = dict(window=window, n_sink=n_sink) if window else {}
    out, lse = c.run(dsa, **kw)
    assert dsa.dsa_read_device_status(c.ws) == (status or dsa.DSA_DEV_BAD_POSITION)
    assert (out[bad] == 0).all() and torch.isneginf(lse[bad]).all()
    c.q_pos[bad] = -1
    ref = c.reference(**kw)
    keep = only if only is not None else list(range(c.T))
    check(out[keep], lse[keep], tuple(x[keep] for x in ref))


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("H", [1, 16, 40])
def test_the_last_token_in_an_unmapped_block(H, block):
    c = leave_row_0(Case([0, 3], [254, 255, 256], H, block=block, lens=[257]))
    c.table[0, 256 // block:] = -1
    run_beside(hide(c, in_order=lambda b, p: p < 256).cuda(), [2])


@pytest.mark.parametrize("block", [7, 16, 64])
@pytest.mark.parametrize("window,n_sink", [(None, 0), (300, 0), (50, 9)])
def test_mapped_rows_that_only_a_token_in_an_unmapped_block_would_see(window, n_sink, block):
    c = leave_row_0(Case([0, 3, 4], [100, 1500, 99, 30], 16, block=block, lens=[1501, 31]))
    c.table[0, 1500 // block:] = -1
    run_beside(hide(c, window or ANY, n_sink, in_order=lambda b, p: p < 1500).cuda(), [1], window, n_sink)


@pytest.mark.parametrize("H", [1, 24])
def test_a_position_past_the_end_of_the_cache(H):
    c = Case([0, 3], [40, 5000, 39], H, lens=[41])
    c.max_kv = 6000
    run_beside(hide(c, in_order=lambda b, p: p < 5000).cuda(), [1])


def test_a_token_in_an_unmapped_block_between_two_windows():
    """Without it the windows of the other two do not meet.  That of the last one
    reaches into the block, so its outputs are unspecified."""
    c = leave_row_0(Case([0, 3], [10, 35, 60], 16, block=16, lens=[61]))
    c.table[0, 2] = -1                                        # 32..47
    hide(c, 30, 0, in_order=lambda b, p: p != 35).cuda()
    run_beside(c, [1], 30, 0, dsa.DSA_DEV_BAD_POSITION | dsa.DSA_DEV_BAD_INDEX, only=[0])


@pytest.mark.parametrize("block", [0, 16])
def test_no_token_in_order(block):
    c = Case([0, 2, 3], [3000, 3001, 20], 16, block=block, lens=[40, 21])
    c.max_kv = 4000
    if block:                                                 # the table covers max_kv positions
        c.table = torch.nn.functional.pad(c.table, (0, 4000 // block - c.table.shape[1]), value=-1)
    run_beside(hide(c, in_order=lambda b, p: p < 3000).cuda(), [0, 1])


def test_an_unmapped_block_that_is_seen_beside_a_gap():
    c = Case([0, 3], [10, 500, 260], 16, block=16, lens=[501])
    c.table[0, 16] = -1                                       # 256..271: the last token's own
    hide(c, 30, 0, in_order=lambda b, p: p != 260).cuda()
    out, lse = c.run(dsa, window=30)
    assert dsa.dsa_read_device_status(c.ws) == dsa.DSA_DEV_BAD_POSITION
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    c.q_pos[2] = -1
    check(out, lse, c.reference(window=30))
    c.table[0, 30] = -1                                       # 480..495: seen from 500
    out, lse = c.run(dsa, window=30)
    assert dsa.dsa_read_device_status(c.ws) == dsa.DSA_DEV_BAD_INDEX
    check(out[:1], lse[:1], tuple(x[:1] for x in c.reference(window=30)))
