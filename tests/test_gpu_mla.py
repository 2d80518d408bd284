"""dsa_mla_attn and dsa_mla_attn_window against their definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402
from _mla_ref import Case, check  # noqa: E402

pytestmark = pytest.mark.gpu


def chunk(lens, per):
    """cu_q and q_pos of the last per[b] tokens of sequences of lens[b] positions."""
    cu, pos = [0], []
    for n, k in zip(lens, per):
        pos += range(n - k, n)
        cu.append(len(pos))
    return cu, pos


def run_and_check(c, **kw):
    attend = {k: kw[k] for k in ("window", "n_sink", "sink_pos0") if k in kw}
    out, lse = c.run(dsa, **kw)
    assert dsa.dsa_read_device_status(c.ws) == 0
    check(out, lse, c.reference(**attend))
    return out, lse


@pytest.mark.parametrize("H", [1, 16, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 16, 127, 128, 129, 300])
def test_one_token(H, n):
    run_and_check(Case(*chunk([n], [1]), H).cuda())


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("H", [5, 33, 64])
def test_ragged_decode(H, tail):
    lens = [1, 500, 64, 3000, 129, 777, 128]
    run_and_check(Case(*chunk(lens, [1] * 7), H, tail).cuda())


@pytest.mark.parametrize("block", [1, 7, 16, 48, 64, 100, 128, 256])
def test_pages(block):
    lens = [300, 1, 129, 515]
    run_and_check(Case(*chunk(lens, [3, 1, 2, 5]), 24, block=block).cuda())


@pytest.mark.parametrize("H", [1, 3, 64, 100, 128])
def test_chunks_of_different_lengths(H):
    lens, per = [700, 40, 0, 333, 1], [130, 40, 0, 7, 1]
    run_and_check(Case(*chunk(lens, per), H).cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_output_types(dtype):
    c = Case(*chunk([900, 260], [4, 3]), 64).cuda()
    run_and_check(c, dtype=dtype)
    out, _ = c.run(dsa, dtype=dtype, lse=False)
    check(out, None, c.reference())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (128, 0), (100, 200), (129, 4), (1000, 64), (2 ** 31 - 1, 5)])
@pytest.mark.parametrize("block", [0, 16, 64])
def test_windows(window, sinks, block):
    lens, per = [900, 1, 411, 130], [9, 1, 140, 130]
    run_and_check(Case(*chunk(lens, per), 16, block=block).cuda(), window=window, n_sink=sinks)


def test_sinks_from_the_first_present_position():
    c = Case(*chunk([900, 700, 50], [3, 2, 5]), 16).cuda()
    a = torch.tensor([130, -7, 2000], dtype=torch.int32, device="cuda")
    run_and_check(c, window=64, n_sink=20, sink_pos0=a)


def test_blocks_out_of_the_window_may_be_unmapped():
    c = Case(*chunk([1000, 600], [4, 1]), 16, block=64).cuda()
    ref = c.reference(window=200, n_sink=10)
    c.table[0, 1:12] = -1                # positions 64..767; the window begins at 797 - 200 + ...
    c.table[1, 1:6] = -1                 # 64..383; window from 400
    out, lse = c.run(dsa, window=200, n_sink=10)
    assert dsa.dsa_read_device_status(c.ws) == 0
    check(out, lse, ref)


def test_positions_in_any_order():
    """Tokens of a tree, all of one sequence: repeated and descending positions."""
    pos = [300, 299, 10, 500, 500, 0, 127, 128, 400]
    run_and_check(Case([0, 9], pos, 40, lens=[501]).cuda())
    run_and_check(Case([0, 9], pos, 40, lens=[501]).cuda(), window=30, n_sink=3)


def test_padding_and_bad_positions():
    cu, pos = [0, 3, 5, 6], [-1, 40, 41, -1, -1, 90]
    c = Case(cu, pos, 48, lens=[42, 3, 91]).cuda()
    run_and_check(c)
    c.q_pos[1] = 10 ** 6                 # out of bounds: flagged, empty
    out, lse = c.run(dsa)
    assert dsa.dsa_read_device_status(c.ws) == dsa.DSA_DEV_BAD_POSITION
    c.q_pos[1] = -1
    check(out, lse, c.reference())
    c.q_pos[1] = -5
    out, lse = c.run(dsa)
    assert dsa.dsa_read_device_status(c.ws) == dsa.DSA_DEV_BAD_POSITION


def test_all_padding():
    c = Case([0, 2, 4], [-1] * 4, 16, lens=[5, 5]).cuda()
    out, lse = run_and_check(c)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_unmapped_blocks_are_flagged():
    c = Case(*chunk([300, 200], [1, 1]), 16, block=64).cuda()
    ref = c.reference()
    c.table[0, 4] = -1                   # the token's own block
    out, lse = c.run(dsa)
    assert dsa.dsa_read_device_status(c.ws) & dsa.DSA_DEV_BAD_POSITION
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    check(out[1:], lse[1:], tuple(x[1:] for x in ref))
    c.table[0, 4], c.table[0, 2] = 0, -1
    out, _ = c.run(dsa)
    assert dsa.dsa_read_device_status(c.ws) == dsa.DSA_DEV_BAD_INDEX
    check(out[1:], None, tuple(x[1:] for x in ref))


def test_rows_behind_the_last_sequence_stay():
    c = Case([0, 2], [40, 41, 9, 9], 16, lens=[42]).cuda()
    ref = c.reference()
    out, lse = c.run(dsa)
    assert (out[2:] == 7).all() and (lse[2:] == 7).all()
    check(out[:2], lse[:2], tuple(x[:2] for x in ref))


def test_sharp_and_growing_scores():
    """Maxima that rise by far more than the rescaling threshold, tile after tile."""
    c = Case(*chunk([1500, 700], [2, 1]), 64, q_size=8.0).cuda()
    c.kv *= torch.linspace(0.1, 4.0, c.rows, device="cuda", dtype=torch.bfloat16)[:, None]
    run_and_check(c)
    c.sm = -c.sm
    run_and_check(c)


def test_equal_scores_give_the_mean():
    c = Case(*chunk([777], [1]), 8).cuda()
    c.q_lat.zero_()
    c.q_rope.zero_()
    out, lse = c.run(dsa, dtype=torch.float32)
    off = int(c.kv_off[0])
    mean = c.kv[off:off + 777, :512].double().mean(0)
    assert (out.double() - mean).abs().max() <= 777 * 2.0 ** -23
    assert (lse - torch.log(torch.tensor(777.0))).abs().max() <= 1e-5


def test_agrees_with_the_sparse_attention_over_every_position():
    c = Case(*chunk([300, 200], [1, 1]), 64).cuda()
    c.kv.nan_to_num_(0.0)
    b = c.batch(dsa)
    idx = torch.full((2, 300), -1, dtype=torch.int32, device="cuda")
    idx[0], idx[1, :200] = torch.arange(300), torch.arange(200)
    so, sl = torch.empty(2, 64, 512, device="cuda"), torch.empty(2, 64, device="cuda")
    dsa.dsa_sparse_mla_attn(c.q_lat, c.q_rope, c.kv, b, idx, c.sm, so, sl, dsa.workspace(dsa.DSA_OP_SPARSE_ATTN, b, H=64, k=300))
    out, lse = c.run(dsa, dtype=torch.float32)
    tol = 2 * c.reference()[2]           # each within its bound of the definition
    assert ((out - so).abs() <= tol).all() and (lse - sl).abs().max() < 1e-4


def test_longer_items_split_among_many_clusters():
    run_and_check(Case(*chunk([20000], [1]), 64).cuda())
    run_and_check(Case(*chunk([9000, 30], [2, 1]), 128).cuda())


def test_cache_beyond_32_bits():
    """Rows whose byte offsets and element offsets pass 2^32."""
    rows = 7_600_000                     # 576 values each: 8.8 GB
    lens, per = [260, 150], [3, 1]
    cu, pos = chunk(lens, per)
    c = Case(cu, pos, 16)
    old, src = c.kv_off.clone(), c.kv
    c.kv_off = torch.tensor([rows - 300, rows - 7_500_000 // 2], dtype=torch.int64)
    c.rows = rows
    c.kv = torch.empty(1)
    c.cuda()
    c.kv = torch.empty(rows, 576, dtype=torch.bfloat16, device="cuda")
    for b, n in enumerate(lens):
        o, d = int(old[b]), int(c.kv_off[b])
        c.kv[d:d + n] = src[o:o + n].cuda()
    run_and_check(c)


def test_one_workspace_for_calls_of_different_batches():
    big = Case(*chunk([700, 300], [40, 20]), 64).cuda()
    small = Case(*chunk([50], [1]), 3, seed=1).cuda()
    ws = dsa.workspace(dsa.DSA_OP_MLA_ATTN, big.batch(dsa), H=64)
    got = [(c, c.run(dsa, ws=ws)) for c in (big, small, big, small)]
    for c, (out, lse) in got:
        check(out, lse, c.reference())


def test_captured_and_replayed_with_other_positions():
    c = Case(*chunk([400, 300], [2, 1]), 64, lens=[600, 600]).cuda()
    c.max_kv = 600
    b = c.batch(dsa)
    ws = dsa.workspace(dsa.DSA_OP_MLA_ATTN, b, H=64)
    out, lse = c.run(dsa, ws=ws)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        dsa.dsa_mla_attn(c.q_lat, c.q_rope, c.kv, b, c.sm, out, lse, ws)
    for pos in ([400, 401, 599], [0, 1, 2], [-1, 5, 300]):
        c.q_pos.copy_(torch.tensor(pos, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check(out, lse, c.reference())


def test_results_do_not_change_between_runs():
    c = Case(*chunk([3000, 1000], [3, 1]), 64).cuda()
    a = c.run(dsa)
    for _ in range(3):
        b = c.run(dsa)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_at_once():
    cs = [Case(*chunk([2000, 90], [3, 1]), 64, seed=s).cuda() for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got.append(c.run(dsa))
    torch.cuda.synchronize()
    for c, (out, lse) in zip(cs, got):
        check(out, lse, c.reference())


def test_a_wait_that_runs_out_is_reported():
    c = Case(*chunk([700], [2]), 64).cuda()
    ref = c.reference()
    ws = dsa.workspace(dsa.DSA_OP_MLA_ATTN, c.batch(dsa), H=64)
    dsa.dsa_set_test_faults(2_000_000, True)
    try:
        c.run(dsa, ws=ws)
        torch.cuda.synchronize()
    finally:
        dsa.dsa_set_test_faults(0, False)
    assert dsa.dsa_read_device_status(ws) & dsa.DSA_DEV_TIMEOUT
    out, lse = c.run(dsa, ws=ws)
    assert dsa.dsa_read_device_status(ws) == 0
    check(out, lse, ref)


@pytest.mark.parametrize("B,H", [(384, 128), (385, 16), (1100, 3)])
def test_many_decoding_sequences(B, H):
    """Up to one thread a sequence the kernel plans for itself; beyond that a plan goes ahead of it."""
    lens = [1 + (37 * b) % 300 for b in range(B)]
    run_and_check(Case(*chunk(lens, [1] * B), H).cuda())


def test_more_items_than_the_plan_has_threads():
    c = Case(*chunk([1300], [1300]), 128).cuda()
    ref = c.reference(window=70)
    out, lse = c.run(dsa, window=70)
    assert dsa.dsa_read_device_status(c.ws) == 0
    check(out, lse, ref)


def test_scale_of_zero_gives_the_mean():
    c = Case(*chunk([130, 64], [2, 1]), 16, block=16).cuda()
    c.sm = 0.0
    run_and_check(c)


def test_queries_of_padding_may_be_anything():
    c = Case([0, 4], [-1, 700, -1, 701], 24).cuda()
    c.q_lat[0], c.q_rope[0] = float("nan"), float("inf")
    c.q_lat[2] = float("-inf")
    run_and_check(c)


@pytest.mark.parametrize("H", [16, 3])
def test_sequence_offsets_that_fall_are_flagged(H):
    c = Case([0, 2, 3], [40, 41, 9], H, lens=[42, 10]).cuda()
    ref = c.reference()
    b, lse = c.batch(dsa), torch.empty(3, H, device="cuda")
    ws = dsa.workspace(dsa.DSA_OP_MLA_ATTN, b, H=H)
    for most in (2, 300):                                     # as decode, and as chunks
        out = torch.full((3, H, 512), 7.0, device="cuda")
        bad = dsa.Batch(torch.tensor([0, 2, 1], dtype=torch.int32, device="cuda"), c.q_pos, c.kv_off, most, c.max_kv, c.rows)
        dsa.dsa_mla_attn(c.q_lat, c.q_rope, c.kv, bad, c.sm, out, lse, ws)
        assert dsa.dsa_read_device_status(ws) == dsa.DSA_DEV_BAD_POSITION
        check(out[:2], lse[:2], tuple(x[:2] for x in ref))
        assert (out[2] == 7).all()
    dsa.dsa_mla_attn(c.q_lat, c.q_rope, c.kv, b, c.sm, out, lse, ws)
    check(out, lse, ref)


@pytest.mark.parametrize("H", [7, 8, 64])
def test_a_few_tokens_a_sequence(H):
    """Sequences of several items each, some without tokens, few enough for the kernel's own plan."""
    lens, per = [300, 5, 0, 513, 40, 0, 129], [9, 5, 0, 4, 1, 0, 20]
    run_and_check(Case(*chunk(lens, per), H).cuda())
    run_and_check(Case(*chunk(lens, per), H, block=16).cuda(), window=100, n_sink=2)


def test_as_many_items_as_threads():
    for tokens in (382, 383, 384):                            # 382 items and their sequence, to 385
        run_and_check(Case(*chunk([tokens, 3], [tokens, 1]), 128).cuda(), window=33, n_sink=1)


@pytest.mark.parametrize("window,sinks", [(130, 0), (37, 150), (300, 17), (257, 300)])
@pytest.mark.parametrize("block", [0, 7, 16, 48, 64, 100, 128])
def test_windows_over_pages_of_any_size(window, sinks, block):
    """Windows and first positions that begin and end inside pages, and meet or not."""
    c = Case(*chunk([777, 300, 520], [5, 2, 3]), 33, block=block).cuda()
    a = torch.tensor([0, 5, 130], dtype=torch.int32, device="cuda")
    run_and_check(c, window=window, n_sink=sinks, sink_pos0=a)
