"""sample against float64: tokens equal, shares within the roundings of one division and one fp32 result."""
import math

import numpy as np
import pytest
import torch

from paged_util import DT, ref_sample
from parity_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def check(x, u, cover=0.9, **kw):
    """x: torch logits on the CPU; kw: numpy settings; cover: the share of rows that can be told apart at least."""
    import block_draft_model_dspark_b200 as dsp
    R, V = x.shape
    dev = {k: torch.from_numpy(v).cuda() for k, v in kw.items()}
    probs = torch.full((R,), -5.0, device="cuda")
    tok = dsp.sample(x.cuda(), torch.from_numpy(u).cuda(), probs=probs, **dev)
    want, prob, margin = ref_sample(x.float().numpy(), u, **kw)
    # 64-bit sums of V terms: u * total is known to V 2^-52 of the total on either side
    sure = margin > V * 2.0 ** -50
    assert sure[u > 0].mean() > cover                 # u = 0 is itself an edge where weights vanish
    got = tok.cpu().numpy()
    assert np.array_equal(got[sure], want[sure]), (np.nonzero(got != want)[0][:5], got[got != want][:5], want[got != want][:5])
    np.testing.assert_allclose(probs.cpu().numpy()[sure], prob[sure], rtol=2.0 ** -23, atol=2.0 ** -149)


def logits(seed, R, V, dt, spread=2.5, peaks=8):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, V)) * spread
    for r in range(R):
        x[r, rng.integers(0, V, peaks)] += 6 + 3 * rng.random(peaks)
    return torch.from_numpy(x.astype(np.float32)).to(DT[dt]), rng


def settings(rng, R):
    pick = lambda t, off, share: np.where(rng.random(R) < share, t, off)  # noqa: E731
    return dict(temperature=pick(0.3 + rng.random(R) * 1.2, 0.0, 0.9).astype(np.float32), top_k=pick(rng.integers(1, 80, R), 0, 0.5).astype(np.int32),
                top_p=pick(0.3 + 0.7 * rng.random(R), 1.0, 0.6).astype(np.float32), min_p=pick(0.2 * rng.random(R), 0.0, 0.4).astype(np.float32))


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("R,V", [(1, 1), (5, 2), (40, 33), (64, 1000), (33, 32003), (20, 50257), (6, 262144)])
def test_sample_matches_reference(dt, R, V):
    x, rng = logits(R * 7 + V, R, V, dt)
    check(x, rng.random(R, dtype=np.float32), **settings(rng, R))
    check(x, rng.random(R, dtype=np.float32))


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p"])
def test_each_filter_alone(name):
    x, rng = logits(1, 200, 3001, "fp32", spread=1.5)
    check(x, rng.random(200, dtype=np.float32), **{name: settings(rng, 200)[name]})


def test_flat_rows_keep_many_candidates():
    """Prefixes of tens of thousands: top-p of a flat row, and a top-k above every short list."""
    x, rng = logits(2, 12, 100003, "fp32", spread=0.5, peaks=1)
    u = rng.random(12, dtype=np.float32)
    check(x, u, top_p=np.full(12, 0.95, np.float32))
    check(x, u, top_k=np.full(12, 60000, np.int32))
    check(x, u, top_k=np.full(12, 60000, np.int32), top_p=np.full(12, 0.9, np.float32), temperature=np.full(12, 0.8, np.float32))
    check(x, u, top_k=np.full(12, 100003, np.int32), min_p=np.full(12, 0.5, np.float32))


@pytest.mark.parametrize("V", [7, 5000, 70001])
def test_ties_go_to_the_lower_index(V):
    """Few distinct values: every boundary falls among equal logits."""
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.integers(0, 4, (30, V)).astype(np.float32))
    x[0] = 1.0
    x[1] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)
    u = rng.random(30, dtype=np.float32)
    check(x, u, temperature=np.full(30, 0.0, np.float32))
    k = rng.integers(1, V + 1, 30).astype(np.int32)
    check(x, u, top_k=k)
    # masses of small integers' weights: an exact edge may fall either way, so p is irrational enough
    check(x, u, top_p=(0.2 + 0.7 * rng.random(30)).astype(np.float32), top_k=k)
    check(x, u, min_p=np.full(30, 0.3, np.float32))


def test_masked_and_special_logits():
    V = 4099
    x, rng = logits(4, 12, V, "fp32")
    inf = float("inf")
    x[0] = -inf                                     # nothing to choose from
    x[1] = -inf
    x[1, 77] = -3.0                                 # one choice
    x[2, ::2] = -inf
    x[3, 5] = float("nan")
    x[4] = float("nan")
    x[5, 9] = inf
    x[6, [9, 4000]] = inf
    x[7] = torch.finfo(torch.float32).min           # a mask's lowest value everywhere: flat
    x[8, 100:] = torch.finfo(torch.float32).min
    x[9] *= 1e30
    u = rng.random(12, dtype=np.float32)
    check(x, u)
    check(x, u, temperature=np.zeros(12, np.float32))
    check(x, u, top_k=np.full(12, 3, np.int32), top_p=np.full(12, 0.7, np.float32))
    check(x, u, top_p=np.full(12, 0.7, np.float32), min_p=np.full(12, 0.01, np.float32))


def test_extreme_settings():
    x, rng = logits(5, 16, 2000, "fp32")
    u = rng.random(16, dtype=np.float32)
    u[:4] = [0.0, np.float32(1) - np.float32(2) ** -24, 0.0, 0.5]
    check(x, u, top_p=np.zeros(16, np.float32))
    check(x, u, min_p=np.ones(16, np.float32))
    check(x, u, top_k=np.ones(16, np.int32))
    check(x, u, temperature=np.full(16, 1e-30, np.float32))
    check(x, u, temperature=np.full(16, 1e30, np.float32))
    check(x, u, top_k=np.full(16, -1, np.int32), top_p=np.full(16, 2.0, np.float32), min_p=np.full(16, -1.0, np.float32))


def test_strided_rows_and_unaligned_starts():
    import block_draft_model_dspark_b200 as dsp
    x, rng = logits(6, 9, 1003, "bf16")
    u = rng.random(9, dtype=np.float32)
    wide = torch.full((9, 1500), 50.0, dtype=torch.bfloat16)
    wide[:, 101:1104] = x
    got = dsp.sample(wide.cuda()[:, 101:1104], torch.from_numpy(u).cuda())
    assert np.array_equal(got.cpu().numpy(), ref_sample(x.float().numpy(), u)[0])
    assert dsp.sample(x.cuda()[:0], torch.zeros(0, device="cuda")).shape == (0,)


@pytest.mark.parametrize("dt,V", [("fp32", 262144), ("bf16", 131072)])
def test_prefixes_that_end_far_down_the_tail(dt, V):
    """top_p near 1: the last part per thousand of the mass is spread over most of the vocabulary."""
    x, rng = logits(7, 12, V, dt)
    u = (1 - 0.002 * rng.random(12)).astype(np.float32)       # and the draw is there too
    for T in (0.6, 1.0, 1.3):
        # cover: an edge lies at most half a token's share away, and at T = 0.6 the shares down there are below
        # exp(-14 / 0.6) = 2^-33.7, less than the 2^-32 (V 2^-50) that sums of V terms may be off: such rows tell nothing
        check(x, u, cover=0.5, temperature=np.full(12, T, np.float32), top_p=np.repeat([0.99, 0.999, 0.9999], 4).astype(np.float32))


def test_more_rows_than_sms():
    """One CTA per row (each pass streams the row), a few per row, and a cluster of CTAs per row draw the same tokens."""
    import block_draft_model_dspark_b200 as dsp
    x, rng = logits(8, 400, 40009, "fp32")
    u = rng.random(400, dtype=np.float32)
    kw = settings(rng, 400)
    check(x, u, **kw)
    dev = {k: torch.from_numpy(v).cuda() for k, v in kw.items()}
    whole = dsp.sample(x.cuda(), torch.from_numpy(u).cuda(), **dev).cpu()
    for n in (1, 7, 60):
        part = dsp.sample(x[:n].cuda(), torch.from_numpy(u[:n]).cuda(), **{k: t[:n].contiguous() for k, t in dev.items()}).cpu()
        assert (part != whole[:n]).sum() <= 0


@pytest.mark.parametrize("R", [3, 200])
def test_top_k_of_every_size(R):
    """Around the list's sizes: a thread's maximum each (512), eight (2048), and beyond."""
    x, rng = logits(9, R, 30011, "fp32")
    u = rng.random(R, dtype=np.float32)
    for k in (1, 2, 511, 512, 513, 1500, 2047, 2048, 2049, 30010):
        check(x, u, top_k=np.full(R, k, np.int32))
    check(x, u, top_k=rng.integers(400, 2300, R).astype(np.int32), top_p=np.full(R, 0.95, np.float32), min_p=np.full(R, 0.001, np.float32))


def test_streamed_rows_on_dirty_shared_memory():
    """Rows that one CTA streams sum weights in their first pass already: the table of powers they read is complete by then,
    whatever the kernel before left in shared memory."""
    import block_draft_model_dspark_b200 as dsp
    R, V = 300, 20011                                             # more rows than places, 80 KB a row: none is kept
    x, rng = logits(10, R, V, "fp32")
    u = rng.random(R, dtype=np.float32)
    table = torch.zeros(R, 1, dtype=torch.int32, device="cuda")
    cache = dsp.PagedKvCache(1, 16, 1, 128, block_table=table, dtype=torch.float16)
    q = torch.full((R * 130, 1, 128), 6e4, dtype=torch.float16, device="cuda")        # as the powers of the table: 1e286
    cu = torch.arange(R + 1, dtype=torch.int32, device="cuda") * 130
    kv = torch.full((R,), 16, dtype=torch.int32, device="cuda")
    xd, ud = x.cuda(), torch.from_numpy(u).cuda()
    for kw in (dict(temperature=np.full(R, 0.9, np.float32)), dict(top_p=np.full(R, 0.9, np.float32))):
        check(x, u, **kw)
        dev = {k: torch.from_numpy(v).cuda() for k, v in kw.items()}
        want, share = dsp.sample(xd, ud, **dev), torch.zeros(R, device="cuda")
        for _ in range(20):
            dsp.attend_paged(q, cache, 0, cu, kv, 130, 1.0)       # fills every SM's shared memory with its queries
            probs = torch.zeros(R, device="cuda")
            got = dsp.sample(xd, ud, probs=probs, **dev)
            assert torch.equal(got, want)
            share = probs if not share.any() else share
            assert torch.equal(probs, share)


@pytest.mark.parametrize("dt,V,near,below", [("fp32", 4_198_401, 4_100_000, 0.998 / 64), ("fp32", 5_100_001, 4_330_000, 0.98 / 64), ("fp16", (1 << 24) - 1, 15_500_000, 9 * 2.0 ** -11)])
def test_millions_of_logits_in_one_bin(dt, V, near, below):
    """Top-p's histogram with millions of entries in the maximum's bin, `below` the maximum, whose places (in 1 / 1024 of a
    bin) come close to 2^32 together or pass it, and a thin tail in which the prefix ends."""
    import block_draft_model_dspark_b200 as dsp
    R = 150                                                       # as few CTAs a row as their slices allow: one, two, four
    rng = np.random.default_rng(V)
    x = torch.empty(V)
    x[:near] = 1.0 - below
    x[77] = 1.0
    x[near:] = torch.from_numpy(0.9 - rng.random(V - near) * (V - near) / (64 * 1500)).float()      # 1500 a bin
    x = x.to(DT[dt]).cuda()
    share = float(torch.exp(x[near:].double() - 1).sum() / torch.exp(x.double() - 1).sum())        # the tail's
    p = (1 - share * rng.uniform(0.03, 0.15, R)).astype(np.float32)
    u = rng.uniform(1 - 2 * share, 1.0, R).astype(np.float32)
    probs = torch.zeros(R, device="cuda")
    tok = dsp.sample(x.expand(R, V).contiguous(), torch.from_numpy(u).cuda(), top_p=torch.from_numpy(p).cuda(), probs=probs).cpu()
    order = torch.argsort(x, descending=True, stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(V, device="cuda")
    # exact sums here: whole numbers of 2^-38 (V of them stay below 2^63). They are off by V 2^-39 at most, the kernel's by its
    # weights (2^-45, twice where a maximum changes) and the additions of a thread's chain, V / 1024 of them, and of the join
    w = torch.round(torch.exp(x.double() - 1) * 2.0 ** 38).long()
    before = (torch.cumsum(w[order], 0) - w[order]).double() * 2.0 ** -38
    total, told = float(w.sum()) * 2.0 ** -38, 0
    off = V * 2.0 ** -38 + 2 * total * ((V / 1024 + 64) * 2.0 ** -53 + 2.0 ** -44)
    for r in range(R):
        n = int((before < float(p[r]) * total).sum())
        c = torch.cumsum(torch.where(rank < n, w, torch.zeros_like(w)), 0).double() * 2.0 ** -38
        want = float(u[r]) * float(c[-1])
        if min(float((before - float(p[r]) * total).abs().min()), float((c - want).abs().min())) < off:
            continue
        told += 1
        at = int((c <= want).sum())
        assert int(tok[r]) == at, (r, int(tok[r]), at)
        prob = math.exp(float(x[at]) - 1) / float(c[-1])
        assert abs(float(probs[r]) - prob) <= 2.0 ** -23 * prob
    assert told > R // 2
