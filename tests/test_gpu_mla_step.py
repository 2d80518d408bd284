"""The calls of a layer together, as a prompt and the tokens after it use them: the
norms of the residual stream and of the latents, the rows into the cache, the tails'
rotation, attention over all rows or through a window."""
import pytest

torch = pytest.importorskip("torch")

import dsa_sparse_attention_score_gb300 as dsa  # noqa: E402
from _mla_ref import attention, check, rows_of  # noqa: E402
from _q8_ref import rotate  # noqa: E402
from test_gpu_norm import check_out, definition  # noqa: E402

pytestmark = pytest.mark.gpu
H, D, EPS, SM, WINDOW, SINKS = 24, 1024, 1e-6, 192 ** -0.5, 40, 3
BF = torch.bfloat16


class Layer:
    """Weights and the cache of one layer."""

    def __init__(self, rows, window, seed):
        g = torch.Generator().manual_seed(seed)
        self.window = window
        self.w_in = (1 + 0.1 * torch.randn(D, generator=g)).to(BF).cuda()
        self.w_lat = (1 + 0.1 * torch.randn(512, generator=g)).to(BF).cuda()
        self.rope = dsa.Rope.make(64)
        self.kv = torch.full((rows, 576), float("nan"), dtype=BF, device="cuda")


class Step:
    """One call of a layer for T tokens: inputs, as projections would leave them, and outputs."""

    def __init__(self, T, seed):
        g = torch.Generator().manual_seed(seed)
        self.x, self.residual, self.proj = (torch.randn(T, n, generator=g).to(BF).cuda() for n in (D, D, 576))
        q = torch.randn(T, H, 576, generator=g).to(BF).cuda()
        self.q_lat, self.q_rope = q[..., :512].contiguous(), q[..., 512:]
        self.h, self.codes = torch.empty_like(self.x), torch.empty(T, D, dtype=torch.uint8, device="cuda")
        self.scale = torch.empty(T, D // 128, device="cuda")
        self.c = torch.empty(T, 512, dtype=BF, device="cuda")
        self.q_turned = torch.empty(T, H, 64, dtype=BF, device="cuda")
        self.out, self.lse = torch.empty(T, H, 512, dtype=BF, device="cuda"), torch.empty(T, H, device="cuda")

    def run(self, layer, batch, ws, page):
        dsa.dsa_rms_norm_q8(self.x, self.residual, self.h, layer.w_in, EPS, self.codes, self.scale)
        dsa.dsa_rms_norm(self.proj[:, :512], None, None, layer.w_lat, EPS, self.c)
        dsa.dsa_kv_append(self.c, self.proj[:, 512:], batch, layer.rope, layer.kv, ws, *page)
        dsa.dsa_rope(self.q_rope, batch.q_pos, layer.rope, self.q_turned)
        if layer.window:
            dsa.dsa_mla_attn_window(self.q_lat, self.q_turned, layer.kv, batch, WINDOW, SINKS, None, SM, self.out, self.lse, ws, *page)
        else:
            dsa.dsa_mla_attn(self.q_lat, self.q_turned, layer.kv, batch, SM, self.out, self.lse, ws, *page)

    def check(self, layer, batch, page):
        pos, cu = batch.q_pos, batch.cu_q.tolist()
        h, y = definition(self.x, self.residual, layer.w_in, EPS)
        assert torch.equal(self.h, h)
        got = self.codes.view(torch.float8_e4m3fn).double().view(-1, D // 128, 128) * self.scale.double()[..., None]
        # half a step of e4m3, or of its least one, beside what y itself is off by
        tol = got.abs().view_as(y) * 2.0 ** -4 + (self.scale.double() * 2.0 ** -10)[..., None].expand_as(got).reshape(y.shape) + y.abs() * 2.0 ** -17
        assert ((got.view_as(y) - y).abs() <= tol).all()
        check_out(self.c, definition(self.proj[:, :512], None, layer.w_lat, EPS)[1])
        freq = layer.rope.inv_freq.cpu().numpy()

        def check_turned(ours, x):
            # float32 products of values in bf16, rounded once
            ref, size = (torch.as_tensor(v).cuda() for v in rotate(x.double().cpu().numpy(), pos.cpu().numpy(), freq, 1.0, True))
            assert ((ours.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + size * 2.0 ** -20).all()

        check_turned(self.q_turned, self.q_rope)
        rows = torch.cat([rows_of(pos[a:b].long(), s, batch.kv_off, page[0], page[1] or 1) for s, (a, b) in enumerate(zip(cu, cu[1:]))])
        assert torch.equal(layer.kv[rows, :512], self.c)
        check_turned(layer.kv[rows, 512:], self.proj[:, 512:])
        window = dict(window=WINDOW, n_sink=SINKS) if layer.window else {}
        check(self.out, self.lse, attention(self.q_lat, self.q_turned, layer.kv, batch.cu_q, pos, batch.kv_off, SM, page[0],
                                            page[1], **window))


@pytest.mark.parametrize("block", [0, 16, 64])
def test_a_prompt_and_the_tokens_after_it(block):
    lens, more, longest = [150, 5, 33], 3, 160
    if block:
        per = -(-longest // block)
        ids = torch.randperm(3 * per, generator=torch.Generator().manual_seed(9)).to(torch.int32).view(3, per).cuda()
        page, rows, off = (ids, block), 3 * per * block, [0, 0, 0]
    else:
        page, rows, off = (None, 0), 3 * longest, [0, longest, 2 * longest]
    layers = [Layer(rows, window, seed) for seed, window in enumerate((False, True))]
    cu = [0, 150, 155, 188]
    prompt = dsa.Batch.from_host(cu, [p for n in lens for p in range(n)], off, rows, max_kv=longest)
    ws = dsa.workspace(dsa.DSA_OP_MLA_ATTN, prompt, H=H)      # serves the appends and the smaller steps as well
    for seed, layer in enumerate(layers):
        s = Step(188, 20 + seed)
        s.run(layer, prompt, ws, page)
        s.check(layer, prompt, page)
    token = dsa.Batch.from_host(range(4), lens, off, rows, max_kv=longest)
    steps = [Step(3, 30 + seed) for seed in range(2)]
    steps[0].run(layers[0], token, ws, page)                  # what the first call of a process sets up
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for s, layer in zip(steps, layers):
            s.run(layer, token, ws, page)
    for n in range(more):
        token.q_pos.copy_(torch.tensor([p + n for p in lens], dtype=torch.int32))
        for s in steps:
            for t in (s.x, s.proj, s.q_lat):
                t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(n)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        for s, layer in zip(steps, layers):
            s.check(layer, token, page)
    assert dsa.dsa_read_device_status(ws) == 0
