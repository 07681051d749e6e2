"""The paged verification step as a target's layer runs it: slots, head norms into the pages, attention, sampling; eager,
captured and replayed with other lengths, on another stream, and two steps at once."""
import numpy as np
import pytest
import torch

from paged_util import HALF, ceil_div, check_attend, ref_attend, ref_page_slots, ref_sample
from parity_util import ensure_built

pytestmark = pytest.mark.gpu

NH, NKV, HD, PAGE, V, LAYERS, TOKENS = 8, 2, 128, 16, 1003, 2, 96


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


class Step:
    """A serving loop's state of B requests: lengths, pages and the buffers of a step of up to TOKENS new tokens."""

    def __init__(self, B=5, max_len=400, seed=0):
        import block_draft_model_dspark_b200 as dsp
        self.dsp, self.B = dsp, B
        g = torch.Generator().manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        pages = B * ceil_div(max_len, PAGE) + 3
        self.cache = dsp.PagedKvCache(pages, PAGE, NKV, HD, batch=B, max_pages=ceil_div(max_len, PAGE), layers=LAYERS, dtype=torch.bfloat16)
        self.cache.k.fill_(float("nan"))                       # rows that no request holds
        self.cache.v.fill_(float("nan"))
        self.free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
        self.count = torch.tensor([pages], **i32)
        self.ctx, self.held, self.new = (torch.zeros(B, **i32) for _ in range(3))
        self.cu, self.slots, self.pos = torch.zeros(B + 1, **i32), torch.zeros(TOKENS, dtype=torch.int64, device="cuda"), torch.zeros(TOKENS, **i32)
        self.x = [torch.zeros(TOKENS, (NH + 2 * NKV) * HD, dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
        self.gain = [(1 + 0.1 * torch.randn(HD, generator=g)).bfloat16().cuda() for _ in range(2)]
        self.freq = dsp.rope_inv_freq(HD, 1e4)
        self.q = [torch.zeros(TOKENS, NH, HD, dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
        self.o = [torch.zeros_like(self.q[0]) for _ in range(LAYERS)]
        self.kv_len = torch.zeros(B, **i32)
        self.ws = dsp.attend_paged_workspace(self.cache, TOKENS, NH, B)
        self.logits = torch.zeros(TOKENS, V, device="cuda")
        self.u, self.T, self.top_p = torch.zeros(TOKENS, device="cuda"), torch.ones(TOKENS, device="cuda"), torch.full((TOKENS,), 0.9, device="cuda")
        self.top_k = torch.full((TOKENS,), 40, **i32)
        self.tok, self.prob = torch.zeros(TOKENS, **i32), torch.zeros(TOKENS, device="cuda")
        self.sws = dsp.sample_workspace(TOKENS, V)

    def feed(self, new, seed):
        g = torch.Generator().manual_seed(seed)
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        for x in self.x:
            x.copy_(torch.randn(x.shape, generator=g))
        self.logits.copy_(torch.randn(self.logits.shape, generator=g) * 3)
        self.u.copy_(torch.rand(TOKENS, generator=g))

    def run(self, stream=None):
        d = self.dsp
        # lengths and pages advance in place: ctx becomes kv_len
        d.page_slots(self.cache, self.ctx, self.new, self.held, self.free, self.count, TOKENS, n_pages_out=self.held, free_count_out=self.count,
                     cu_new=self.cu, kv_len=self.ctx, slots=self.slots, positions=self.pos, stream=stream)
        for l in range(LAYERS):
            q, k, v = (t.unflatten(1, (-1, HD)) for t in self.x[l].split([NH * HD, NKV * HD, NKV * HD], 1))
            d.norm_rope_paged(q, k, v, *self.gain, self.freq, self.pos, self.slots, self.cache, l, v_norm=True, q_out=self.q[l], stream=stream)
            d.attend_paged(self.q[l], self.cache, l, self.cu, self.ctx, TOKENS, HD ** -0.5, out=self.o[l], ws=self.ws, stream=stream)
        d.sample(self.logits, self.u, self.T, self.top_k, self.top_p, tokens=self.tok, probs=self.prob, ws=self.sws, stream=stream)

    def outputs(self):
        n = int(self.cu[-1])
        return [t.clone() for t in (self.ctx, self.held, self.count, self.cu, self.slots, self.pos, self.cache.block_table, self.tok, self.prob)] + \
            [t[:n].clone() for t in self.q + self.o]


def check_step(s, before, new, seed):
    """The step's outputs against the formulas, from the lengths and pages before it."""
    ctx, held, free, count, table = before
    want = ref_page_slots(ctx, new, held, free, count, table, PAGE, TOKENS)
    got = (s.held.tolist(), int(s.count), s.cu.tolist(), s.ctx.tolist(), s.slots.tolist(), s.pos.tolist())
    assert got == tuple(want[:6]) and np.array_equal(s.cache.block_table.cpu().numpy(), want[6])
    n, slots = want[2][-1], torch.tensor(want[4][:want[2][-1]])
    ang = torch.outer(torch.tensor(want[5][:n], dtype=torch.float64), s.freq.cpu())[:, None]
    for l in range(LAYERS):
        x = s.x[l][:n].double().cpu().unflatten(1, (-1, HD))
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        rope = lambda y: torch.cat([y[..., :HD // 2] * ang.cos() - y[..., HD // 2:] * ang.sin(), y[..., HD // 2:] * ang.cos() + y[..., :HD // 2] * ang.sin()], -1)  # noqa: E731
        rows = [rope(x[:, :NH] * s.gain[0].double().cpu()), rope(x[:, NH:NH + NKV] * s.gain[1].double().cpu()), x[:, NH + NKV:]]
        have = [s.q[l][:n], s.cache.k[l].view(-1, NKV, HD)[slots.cuda()], s.cache.v[l].view(-1, NKV, HD)[slots.cuda()]]
        for a, b in zip(have, rows):
            # one rounding to bf16; the 32-bit operations (HD squares, root, gain, angle, turn) are far below: 2^-14 of a
            # pair's size (at most 2 max|y| over a head) covers them
            assert bool(((a.double().cpu() - b).abs() <= HALF[torch.bfloat16] * b.abs() + 2.0 ** -14 * b.abs().amax(-1, keepdim=True)).all())
        ref = ref_attend(s.q[l][:n], s.cache, l, new, want[3], HD ** -0.5, True, 0)
        check_attend(s.o[l][:n], None, ref, torch.bfloat16, max(want[3]), (l, new))
    tok, prob, margin = ref_sample(s.logits.cpu().numpy(), s.u.cpu().numpy(), s.T.cpu().numpy(), s.top_k.cpu().numpy(), s.top_p.cpu().numpy())
    sure = margin > V * 2.0 ** -45                             # weights are within 2^-45
    assert np.array_equal(s.tok.cpu().numpy()[sure], tok[sure])
    np.testing.assert_allclose(s.prob.cpu().numpy()[sure], prob[sure], rtol=2.0 ** -23)
    assert s.cache.read_status() == 0


def lengths(s):
    return s.ctx.tolist(), s.held.tolist(), s.free.cpu().numpy(), int(s.count), s.cache.block_table.cpu().numpy()


STEPS = [[17, 1, 0, 40, 9], [1, 1, 1, 1, 1], [0, 33, 5, 0, 2], [17, 17, 17, 17, 17]]


def test_steps_match_the_formulas():
    s = Step()
    for i, new in enumerate(STEPS):
        before = lengths(s)
        s.feed(new, i)
        s.run()
        check_step(s, before, new, i)


def test_replayed_steps_equal_eager_ones():
    a, b = Step(), Step()
    side = torch.cuda.Stream()
    a.feed([0] * 5, 9)                                         # a first call outside the graph (an empty step)
    a.run()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.run()
    for i, new in enumerate(STEPS):
        for s in (a, b):
            s.feed(new, i)
        graph.replay()
        b.run()
        for x, y in zip(a.outputs(), b.outputs()):
            assert torch.equal(x, y)
    assert a.cache.read_status() == 0


def test_two_steps_on_two_streams():
    a, b, c = Step(seed=1), Step(seed=2), (Step(seed=1), Step(seed=2))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, new in enumerate(STEPS):
        for s in (a, b) + c:
            s.feed(new, i)
        torch.cuda.synchronize()
        a.run(stream=streams[0])                               # by the argument, beside the other by the current stream
        with torch.cuda.stream(streams[1]):
            b.run()
        torch.cuda.synchronize()
        for s in c:
            s.run()
        for s, t in zip((a, b), c):
            for x, y in zip(s.outputs(), t.outputs()):
                assert torch.equal(x, y)


def test_a_refused_step_changes_nothing():
    s = Step()
    s.feed([17, 1, 0, 40, 9], 0)
    s.run()
    kept = [t.clone() for t in (s.ctx, s.held, s.count, s.cache.block_table, s.cache.k, s.cache.v)]
    s.feed([60, 60, 0, 0, 0], 1)                               # more tokens than the step has room for
    s.o[0].fill_(3.0)
    s.run()
    assert s.cache.read_status() == s.dsp.DSPARK_DEV_CAPACITY
    now = (s.ctx, s.held, s.count, s.cache.block_table)
    for x, y in zip(now, kept):
        assert torch.equal(x, y)
    assert torch.equal(s.cache.k.isnan(), kept[4].isnan()) and torch.equal(s.cache.k.nan_to_num(), kept[4].nan_to_num())
    assert bool((s.o[0] == 3.0).all()) and bool((s.slots == -1).all())


def test_results_do_not_change_from_run_to_run():
    """A long request split over every SM: the pieces are joined in one order."""
    import block_draft_model_dspark_b200 as dsp
    g = torch.Generator(device="cuda").manual_seed(4)
    cache = dsp.PagedKvCache(600, 16, 2, 256, block_table=torch.randperm(600, generator=g, device="cuda").to(torch.int32)[None].contiguous(),
                             k=torch.randn(1, 600, 16, 2, 256, generator=g, device="cuda").half(), v=torch.randn(1, 600, 16, 2, 256, generator=g, device="cuda").half())
    q = torch.randn(17, 16, 256, generator=g, device="cuda").half()
    cu, kv = torch.tensor([0, 17], dtype=torch.int32, device="cuda"), torch.tensor([9555], dtype=torch.int32, device="cuda")
    outs = [dsp.attend_paged(q, cache, 0, cu, kv, 17, 0.06) for _ in range(6)]
    assert all(torch.equal(outs[0], o) for o in outs[1:]) and cache.read_status() == 0


def test_calls_on_the_tensors_device_and_stream_own_their_memory():
    """Outputs and workspaces that a call allocates for another stream are that stream's."""
    import block_draft_model_dspark_b200 as dsp
    side = torch.cuda.Stream()
    x = torch.randn(4, 5000, device="cuda")
    u = torch.rand(4, device="cuda")
    want = dsp.sample(x, u)
    torch.cuda.synchronize()
    for _ in range(20):
        got = dsp.sample(x, u, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
