"""page_slots against plain loops: exact, with ragged and empty requests, odd page sizes, in-place outputs,
refusals that leave everything as it was, and pages outside the pool."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from paged_util import ceil_div, ref_page_slots
from parity_util import ensure_built

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def case(seed, B, page, ctx_hi, new_hi, extra_held=0):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, B).tolist()
    new = rng.integers(0, new_hi + 1, B).tolist()
    if B > 2:
        ctx[0], new[1], ctx[2], new[2] = 0, 0, 0, 0
    held = [ceil_div(c, page) + int(rng.integers(0, extra_held + 1)) for c in ctx]
    width = max([ceil_div(c + n, page) for c, n in zip(ctx, new)] + held + [1])
    need = sum(max(0, ceil_div(c + n, page) - h) for c, n, h in zip(ctx, new, held))
    pages = sum(held) + need + 5
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    return ctx, new, held, order[at:].copy(), table, pages


def cache_of(table, pages, page):
    import block_draft_model_dspark_b200 as dsp
    return dsp.PagedKvCache(pages, page, 1, 16, block_table=torch.from_numpy(table.copy()).cuda())


def dev(v, dt=torch.int32):
    return torch.tensor(v, dtype=dt, device="cuda")


@pytest.mark.parametrize("B,page,ctx_hi,new_hi,held", [(1, 64, 4096, 17, 0), (3, 1, 5, 4, 2), (37, 16, 300, 40, 3), (64, 24, 1000, 129, 0),
                                                       (1000, 16, 100, 9, 1), (4096, 64, 200, 3, 0), (5, 128, 0, 20000, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_slots_match_loops(B, page, ctx_hi, new_hi, held, in_place):
    import block_draft_model_dspark_b200 as dsp
    ctx, new, hp, free, table, pages = case(B * 7 + page, B, page, ctx_hi, new_hi, held)
    T = sum(new) + 13
    cache = cache_of(table, pages, page)
    c, n, h, f, k = dev(ctx), dev(new), dev(hp), torch.from_numpy(free).cuda(), dev([len(free)])
    kw = dict(n_pages_out=h, free_count_out=k, kv_len=c) if in_place else {}
    cu, kv, slots, pos, hp2, k2 = dsp.page_slots(cache, c, n, h, f, k, T, **kw)
    want = ref_page_slots(ctx, new, hp, free.tolist(), len(free), table, page, T)
    assert hp2.tolist() == want[0] and k2.tolist() == [want[1]] and cu.tolist() == want[2] and kv.tolist() == want[3]
    assert slots.tolist() == want[4] and pos.tolist() == want[5]
    assert np.array_equal(cache.block_table.cpu().numpy(), want[6])
    assert cache.read_status() == 0
    assert f.cpu().numpy().tolist() == free.tolist()


def test_page_slots_step_after_step():
    """The counts of one call feed the next; a request that shrank (rejected tokens) keeps its pages."""
    import block_draft_model_dspark_b200 as dsp
    rng = np.random.default_rng(5)
    B, page, pages = 9, 16, 200
    table = np.full((B, 20), -1, np.int32)
    free = rng.permutation(pages).astype(np.int32)
    cache = cache_of(table, pages, page)
    ctx, hp, count = [0] * B, [0] * B, pages
    h, f, k = dev(hp), torch.from_numpy(free).cuda(), dev([count])
    for step in range(6):
        new = rng.integers(0, 30, B).tolist()
        cu, kv, slots, pos, _, _ = dsp.page_slots(cache, dev(ctx), dev(new), h, f, k, 400, n_pages_out=h, free_count_out=k)
        want = ref_page_slots(ctx, new, hp, free.tolist(), count, table, page, 400)
        assert slots.tolist() == want[4] and h.tolist() == want[0] and k.tolist() == [want[1]]
        hp, count, table = want[0], want[1], want[6]
        ctx = [c + int(rng.integers(0, n + 1)) for c, n in zip(ctx, new)]      # some of the new tokens stay
    assert cache.read_status() == 0


@pytest.mark.parametrize("why", ["pages", "tokens", "negative", "table", "count", "ctx"])
def test_page_slots_refusals_change_nothing(why):
    import block_draft_model_dspark_b200 as dsp
    ctx, new, hp, free, table, pages = case(11, 20, 16, 300, 40)
    T, count = sum(new), len(free)
    if why == "pages":
        count = sum(max(0, ceil_div(c + n, 16) - x) for c, n, x in zip(ctx, new, hp)) - 1
    elif why == "tokens":
        T -= 1
    elif why == "negative":
        new[3] = -1
    elif why == "ctx":
        ctx[19] = -5
    elif why == "table":
        new[4] = table.shape[1] * 16 - ctx[4] + 1
        T += 10000
    elif why == "count":
        count = len(free) + 1
    cache = cache_of(table, pages, 16)
    h, k = dev(hp), dev([count])
    cu, kv, slots, pos, hp2, k2 = dsp.page_slots(cache, dev(ctx), dev(new), h, torch.from_numpy(free).cuda(), k, T)
    assert cu.tolist() == [0] * 21 and set(slots.tolist()) == {-1} and kv.tolist() == ctx
    assert hp2.tolist() == hp and k2.tolist() == [count]
    assert np.array_equal(cache.block_table.cpu().numpy(), table)
    assert cache.read_status() == dsp.DSPARK_DEV_CAPACITY and cache.read_status() == 0


def test_page_slots_bad_page_gives_no_slot():
    import block_draft_model_dspark_b200 as dsp
    table = np.array([[3, 99, -1]], np.int32)                 # page 99 is outside the pool of 10
    cache = cache_of(table, 10, 16)
    cu, kv, slots, pos, _, _ = dsp.page_slots(cache, dev([10]), dev([16]), dev([2]), dev([4]), dev([1]), 16)
    assert slots.tolist() == [3 * 16 + 10 + i for i in range(6)] + [-1] * 10
    assert cache.read_status() == dsp.DSPARK_DEV_BAD_PAGE


def test_many_tokens_over_a_cluster():
    """Sizes at which one, several and sixteen CTAs share the fill, in place."""
    import block_draft_model_dspark_b200 as dsp
    for seed, B, new_hi, pad in ((40, 3, 1000, 0), (41, 700, 40, 7), (42, 4096, 30, 1), (43, 2, 60000, 13)):
        ctx, new, held, free, table, pages = case(seed, B, 16, 300, new_hi)
        total = sum(new) + pad
        cache = cache_of(table, pages, 16)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        c, n, h, cnt = i32(ctx), i32(new), i32(held), i32([len(free)])
        cu, kv, slots, pos, _, _ = dsp.page_slots(cache, c, n, h, torch.from_numpy(free).cuda(), cnt, total, n_pages_out=h, free_count_out=cnt, kv_len=c)
        want = ref_page_slots(ctx, new, held, free, len(free), table, 16, total)
        assert h.tolist() == want[0] and int(cnt) == want[1] and cu.tolist() == want[2] and c.tolist() == want[3]
        assert slots.tolist() == want[4] and pos.tolist() == want[5] and np.array_equal(cache.block_table.cpu().numpy(), want[6])
        assert cache.read_status() == 0


@pytest.mark.parametrize("B", [3055, 3056, 3071, 3080])
def test_tables_around_the_default_shared_memory(B):
    """The largest batches that fit it and the first that do not, each as the first call of a process (the opt-in to more
    stays with the kernel once it is made)."""
    code = ("import torch, block_draft_model_dspark_b200 as dsp\n"
            f"B = {B}\n"
            "i32 = dict(dtype=torch.int32, device='cuda')\n"
            "cache = dsp.PagedKvCache(B, 16, 1, 16, batch=B, max_pages=1)\n"
            "one, none = torch.ones(B, **i32), torch.zeros(B, **i32)\n"
            "cu, kv, slots, pos, held, count = dsp.page_slots(cache, none, one, none, torch.arange(B, **i32), torch.tensor([B], **i32), B)\n"
            "assert cu.tolist() == list(range(B + 1)) and slots.tolist() == [16 * (B - 1 - i) for i in range(B)] and int(count) == 0\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_page_slots_bad_page_without_a_new_token_is_reported():
    """Pages that a request takes for rows it has cached already: a number outside the pool is reported too."""
    import block_draft_model_dspark_b200 as dsp
    cache = cache_of(np.full((1, 3), -1, np.int32), 10, 16)
    cu, kv, slots, pos, held, count = dsp.page_slots(cache, dev([40]), dev([1]), dev([0]), dev([2, 5, 77]), dev([3]), 4)
    assert held.tolist() == [3] and count.tolist() == [0] and slots.tolist() == [2 * 16 + 8, -1, -1, -1]
    assert cache.read_status() == dsp.DSPARK_DEV_BAD_PAGE


def test_pages_of_finished_requests_come_back():
    """Requests that end push their pages onto the free stack: every page belongs to one request or to the stack."""
    import block_draft_model_dspark_b200 as dsp
    rng = np.random.default_rng(50)
    B, pages = 6, 60
    cache = dsp.PagedKvCache(pages, 16, 1, 16, batch=B, max_pages=30)
    free, count = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda(), dev([pages])
    ctx, held = dev([0] * B), dev([0] * B)
    for step in range(12):
        new = dev(rng.integers(0, 40, B).tolist())
        dsp.page_slots(cache, ctx, new, held, free, count, 40 * B, n_pages_out=held, free_count_out=count, kv_len=ctx)
        assert cache.read_status() == 0
        ctx -= torch.minimum(new, dev(rng.integers(0, 5, B).tolist()))
        b = int(torch.argmax(ctx))                                # the longest ends
        n, c = int(held[b]), int(count)
        free[c:c + n] = cache.block_table[b, :n]
        count += n
        held[b] = 0
        ctx[b] = 0
        owned = [int(p) for i in range(B) for p in cache.block_table[i, :int(held[i])]]
        assert sorted(owned + free[:int(count)].tolist()) == list(range(pages))
