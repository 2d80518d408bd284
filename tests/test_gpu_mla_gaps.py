"""Attention through a window over tokens that leave positions between their windows
unseen: those hold NaN or are unmapped, and neither the outputs nor the status know of
it."""
import math

import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402
from _mla_ref import Case, check, rows_of  # noqa: E402

pytestmark = pytest.mark.gpu
ANY = 2 ** 31 - 1


def seen(c, b, window, n_sink, a, in_order):
    """The positions of sequence b that some token in order sees."""
    s = set()
    for t in range(int(c.cu_q[b]), int(c.cu_q[b + 1])):
        p = int(c.q_pos[t])
        if p >= 0 and in_order(b, p):
            s |= set(range(max(0, p - window + 1), p + 1)) | set(range(a[b], min(a[b] + n_sink, p + 1)))
    return sorted(s)


def hide(c, window=ANY, n_sink=0, a=None, in_order=lambda b, p: True):
    """NaN into every row that no token sees (before the case is on the GPU)."""
    a = a or [0] * c.B
    rows = [rows_of(torch.tensor(s), b, c.kv_off, c.table, c.block) for b in range(c.B) if (s := seen(c, b, window, n_sink, a, in_order))]
    unseen = torch.ones(c.rows, dtype=torch.bool)
    unseen[torch.cat(rows)] = False
    c.kv[unseen] = math.nan
    return c


def unmap(c, window, n_sink, a=None):
    """No block for positions of which no token sees any."""
    for b in range(c.B):
        kept = {p // c.block for p in seen(c, b, window, n_sink, a or [0] * c.B, lambda b, p: True)}
        for k in range(c.table.shape[1]):
            if k not in kept:
                c.table[b, k] = -1
    return c


# positions of a sequence's tokens, and a window that leaves gaps between them
SPREADS = [([10, 500], 30), ([300, 299, 10, 500, 500, 0, 127, 128, 400], 30), ([100, 101, 102] + [-1] * 5 + [300, 301], 20),
           ([50, 3000, 1500], 40), ([5, 7, 9, 200, 202], 1), (list(range(4019, 0, -40)), 16), ([700, 20, -1, 21, 699, 350], 129)]


@pytest.mark.parametrize("block", [0, 7, 16, 48, 64])
@pytest.mark.parametrize("H", [1, 16, 40])
@pytest.mark.parametrize("spread", range(len(SPREADS)))
def test_positions_between_windows_may_hold_anything(spread, H, block):
    pos, window = SPREADS[spread]
    n_sink = (0, 3, 20)[spread % 3]
    c = Case([0, len(pos), len(pos) + 2], pos + [60, 61], H, block=block, lens=[max(pos) + 1, 62])
    hide(c, window, n_sink)
    if block:
        unmap(c, window, n_sink)
    c.cuda()
    out, lse = c.run(dsa, window=window, n_sink=n_sink)
    assert dsa.dsa_read_device_status(c.ws) == 0
    check(out, lse, c.reference(window=window, n_sink=n_sink))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gaps_and_first_present_positions(dtype):
    """First positions that end inside a gap, in both output types."""
    pos, a = [900, 30, 200, 31, 640], [130, 40]
    c = Case([0, 5, 7], pos + [500, 41], 24, block=16, lens=[901, 501])
    unmap(hide(c, 25, 18, a), 25, 18, a).cuda()
    s0 = torch.tensor(a, dtype=torch.int32, device="cuda")
    out, lse = c.run(dsa, window=25, n_sink=18, sink_pos0=s0, dtype=dtype)
    assert dsa.dsa_read_device_status(c.ws) == 0
    check(out, lse, c.reference(window=25, n_sink=18, sink_pos0=s0))
