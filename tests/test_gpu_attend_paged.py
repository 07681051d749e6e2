"""attend_paged against the formula in float64: types, head layouts, page sizes, lengths, masks that leave
rows empty, garbage in rows nobody sees, strides, bad pages, and rows behind the last request."""
import numpy as np
import pytest
import torch

from paged_util import DT, check_attend, make_paged, ref_attend
from parity_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def run(seed, new, kv_len, nH, nKv, hd, page, dt, causal=True, window=0, scale=None, layers=1, layer=0, pad=3):
    import block_draft_model_dspark_b200 as dsp
    rng = np.random.default_rng(seed)
    dtype = DT[dt]
    cache = make_paged(rng, kv_len, page, nKv, hd, dtype, layers=layers)
    T = sum(new)
    scale = hd ** -0.5 if scale is None else scale
    q = torch.from_numpy(rng.standard_normal((T + pad, nH, hd)).astype(np.float32)).to(dtype).cuda()
    q[T:] = float("nan")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    kv = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    out = torch.full((T + pad, nH, hd), 3.0, dtype=dtype, device="cuda")
    lse = torch.full((T + pad, nH), 3.0, device="cuda")
    dsp.attend_paged(q, cache, layer, cu, kv, max(new + [0]), scale, causal=causal, window=window, out=out, lse=lse)
    assert cache.read_status() == 0
    ref = ref_attend(q[:T], cache, layer, new, kv_len, scale, causal, window)
    check_attend(out[:T], lse[:T], ref, dtype, max(kv_len + [1]), (new, kv_len))
    assert bool((out[T:] == 3.0).all()) and bool((lse[T:] == 3.0).all())      # rows of no request


# head layouts: (n_heads, n_kv, head_dim)
LAYOUTS = [(16, 2, 256), (8, 8, 128), (6, 2, 64), (5, 1, 192), (32, 2, 128)]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("nH,nKv,hd", LAYOUTS)
def test_ragged_batches(dt, nH, nKv, hd):
    run(1, [1, 17, 0, 3, 40], [1, 100, 65, 3, 333], nH, nKv, hd, 16, dt)


@pytest.mark.parametrize("nH,nKv,hd,page", [(4, 1, 64, 16), (3, 3, 80, 16), (4, 2, 32, 3), (2, 1, 256, 1)])
def test_fp32_and_odd_shapes(nH, nKv, hd, page):
    run(2, [5, 1, 2], [50, 33, 2], nH, nKv, hd, page, "fp32")
    run(2, [5, 1, 2], [50, 33, 2], nH, nKv, hd, page, "bf16", window=7)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_page_sizes_and_pages_ending_in_a_tile(page):
    for kv in ([1], [63], [64], [65], [127, 128, 129], [255, 257, 511]):
        run(3 + page, [1] * len(kv), kv, 4, 2, 128, page, "bf16")
        run(4 + page, [min(k, 9) for k in kv], kv, 4, 2, 64, page, "fp16")


@pytest.mark.parametrize("window", [1, 5, 64, 200])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(window, causal):
    run(5, [30, 1, 130], [300, 90, 130], 4, 2, 128, 16, "bf16", causal=causal, window=window)
    run(6, [30, 1, 130], [300, 90, 130], 4, 2, 256, 32, "fp16", causal=causal, window=window)


def test_not_causal():
    run(7, [30, 1, 150], [300, 90, 150], 6, 2, 128, 16, "bf16", causal=False)
    run(8, [16, 3], [700, 90], 16, 2, 256, 64, "fp16", causal=False)


@pytest.mark.parametrize("hd", [64, 256])
def test_rows_that_see_no_key(hd):
    """Fewer keys than new tokens: the first queries sit before key 0; and a request without keys."""
    run(9, [10, 4, 300, 2], [4, 0, 140, 5], 4, 2, hd, 16, "bf16")
    run(9, [10, 4, 300, 2], [4, 0, 140, 5], 4, 2, hd, 16, "fp16", window=3)


@pytest.mark.parametrize("nH,nKv,hd", [(4, 2, 128), (8, 1, 256), (2, 2, 64)])
def test_long_contexts_and_chunks(nH, nKv, hd):
    run(10, [1, 2], [5000, 9001], nH, nKv, hd, 16, "bf16")
    run(11, [300], [1500], nH, nKv, hd, 64, "fp16")
    run(12, [257, 5, 129], [257, 2000, 700], nH, nKv, hd, 32, "bf16")


def test_wide_groups():
    run(13, [3, 9], [200, 70], 64, 1, 64, 16, "bf16")
    run(14, [1, 2], [200, 70], 128, 1, 128, 16, "fp16")
    run(15, [2], [40], 130, 1, 64, 16, "bf16")


def test_large_scores():
    """Scores far apart: the running maximum moves, the softmax is nearly one-hot."""
    run(16, [20, 1], [700, 900], 4, 2, 128, 16, "fp16", scale=3.0)
    run(17, [140], [700], 4, 2, 128, 16, "bf16", scale=8.0)


def test_layers_and_many_requests():
    run(18, [1] * 200, list(range(1, 201)), 4, 1, 64, 16, "bf16", layers=3, layer=2)
    run(19, [2, 0, 1] * 60, [40, 0, 7] * 60, 2, 1, 128, 8, "fp16", layers=2, layer=1)


def test_strided_queries_and_outputs():
    import block_draft_model_dspark_b200 as dsp
    rng = np.random.default_rng(20)
    new, kv_len, nH, nKv, hd = [7, 140], [50, 300], 4, 2, 128
    cache = make_paged(rng, kv_len, 16, nKv, hd, torch.bfloat16)
    T = sum(new)
    wide = torch.from_numpy(rng.standard_normal((T, (nH + 2 * nKv) * hd)).astype(np.float32)).bfloat16().cuda()
    q = wide[:, :nH * hd].unflatten(1, (nH, hd))
    big = torch.full((T, nH + 1, hd), 2.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 7, 147], dtype=torch.int32, device="cuda")
    dsp.attend_paged(q, cache, 0, cu, torch.tensor(kv_len, dtype=torch.int32, device="cuda"), 140, 0.1, out=big[:, :nH])
    check_attend(big[:, :nH], None, ref_attend(q, cache, 0, new, kv_len, 0.1, True, 0), torch.bfloat16, 300, "strided")
    assert bool((big[:, nH] == 2.0).all())


@pytest.mark.parametrize("hd,page", [(128, 16), (256, 64), (48, 16)])
def test_bad_pages_and_lengths_are_reported(hd, page):
    """A page outside the pool reads as zeros (score 0, value 0); a length past the table is clamped."""
    import block_draft_model_dspark_b200 as dsp
    rng = np.random.default_rng(21)
    kv_len = [3 * page + 5, 40]
    cache = make_paged(rng, kv_len, page, 2, hd, torch.float16)
    q = torch.from_numpy(rng.standard_normal((2, 4, hd)).astype(np.float32)).half().cuda()
    cu, kv = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    for bad in (-1, cache.num_pages, 2 ** 31 - 1):
        good = int(cache.block_table[0, 1])
        cache.block_table[0, 1] = bad
        out = dsp.attend_paged(q, cache, 0, cu, kv, 1, 0.1)
        assert cache.read_status() == dsp.DSPARK_DEV_BAD_PAGE
        cache.block_table[0, 1] = good
        k0, v0 = cache.k.clone(), cache.v.clone()
        cache.k[0, good] = 0
        cache.v[0, good] = 0
        check_attend(out, None, ref_attend(q, cache, 0, [1, 1], kv_len, 0.1, True, 0), torch.float16, 200, bad)
        cache.k.copy_(k0)
        cache.v.copy_(v0)
    kv[1] = cache.max_pages * page + 1
    cache.block_table[1] = cache.block_table[0, 0]
    cache.k[0, int(cache.block_table[0, 0])] = 0.5
    cache.v[0, int(cache.block_table[0, 0])] = 0.25
    out = dsp.attend_paged(q, cache, 0, cu, kv, 1, 0.1)
    assert cache.read_status() == dsp.DSPARK_DEV_BAD_LENGTH
    assert bool((out[1] == 0.25).all())


def test_no_tokens_or_requests():
    import block_draft_model_dspark_b200 as dsp
    cache = dsp.PagedKvCache(4, 16, 1, 64, batch=2, max_pages=2)
    q = torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda")
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert dsp.attend_paged(q, cache, 0, z, z[:2], 0, 1.0).shape == (0, 2, 64)
    out = torch.full((3, 2, 64), 2.0, dtype=torch.float16, device="cuda")
    dsp.attend_paged(torch.zeros_like(out), cache, 0, z[:1], z[:0], 0, 1.0, out=out)
    dsp.attend_paged(torch.zeros_like(out), cache, 0, z, z[:2], 5, 1.0, out=out)
    assert bool((out == 2.0).all()) and cache.read_status() == 0


def test_lengths_that_cannot_be_are_reported():
    """Negative lengths count as 0, offsets past the tokens as their end; rows that belong to nobody stay."""
    import block_draft_model_dspark_b200 as dsp
    rng = np.random.default_rng(30)
    for hd, dt in ((128, torch.bfloat16), (256, torch.float16), (64, torch.float32)):
        cache = make_paged(rng, [40, 50], 16, 2, hd, dt)
        q = torch.from_numpy(rng.standard_normal((6, 4, hd)).astype(np.float32)).to(dt).cuda()
        good = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
        for cu, kv in (([0, 2, 4], [-5, 50]), ([0, 2, 9], [40, 50])):
            out = torch.full((6, 4, hd), 2.0, dtype=dt, device="cuda")
            dsp.attend_paged(q, cache, 0, torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.tensor(kv, dtype=torch.int32, device="cuda"), 5, 0.1, out=out)
            status = cache.read_status()
            if kv[0] < 0:
                assert status == dsp.DSPARK_DEV_BAD_LENGTH and bool((out[:2] == 0).all()) and bool((out[4:] == 2.0).all())
                ref = ref_attend(q[2:4], make_view(cache, 1), 0, [2], [50], 0.1, True, 0)
                check_attend(out[2:4], None, ref, dt, 50, "the other request")
            elif dt is not torch.float32:
                assert status == dsp.DSPARK_DEV_BAD_LENGTH
        out = torch.full((6, 4, hd), 2.0, dtype=dt, device="cuda")
        dsp.attend_paged(q, cache, 0, good, torch.tensor([40, 50], dtype=torch.int32, device="cuda"), 2, 0.1, out=out)
        assert cache.read_status() == 0 and bool((out[4:] == 2.0).all())


def make_view(cache, b):
    """The cache as request b sees it."""
    import block_draft_model_dspark_b200 as dsp
    return dsp.PagedKvCache(cache.num_pages, cache.page_size, cache.n_kv, cache.head_dim, block_table=cache.block_table[b:b + 1].contiguous(), k=cache.k, v=cache.v)


@pytest.mark.parametrize("hd,page", [(64, 16), (128, 32)])
def test_as_many_requests_as_a_call_takes(hd, page):
    new = [(i * 7) % 3 for i in range(4096)]
    run(31, new, [n + (i * 13) % 40 for i, n in enumerate(new)], 2, 1, hd, page, "bf16")


def test_a_window_wider_than_the_request_is_none():
    import block_draft_model_dspark_b200 as dsp
    rng = np.random.default_rng(32)
    cache = make_paged(rng, [300, 90], 16, 2, 128, torch.bfloat16)
    q = torch.from_numpy(rng.standard_normal((40, 4, 128)).astype(np.float32)).bfloat16().cuda()
    cu, kv = torch.tensor([0, 33, 40], dtype=torch.int32, device="cuda"), torch.tensor([300, 90], dtype=torch.int32, device="cuda")
    for causal in (True, False):
        want = dsp.attend_paged(q, cache, 0, cu, kv, 33, 0.1, causal=causal)
        for window in (320, 1 << 20, 2 ** 31 - 1):
            assert torch.equal(dsp.attend_paged(q, cache, 0, cu, kv, 33, 0.1, causal=causal, window=window), want)


def test_max_new_only_chooses_tiles():
    """The bound on a request's new tokens may be loose: results stay within their roundings."""
    for max_new in (1, 500):
        import block_draft_model_dspark_b200 as dsp
        rng = np.random.default_rng(33)
        new, kv_len = [70, 1, 16], [200, 90, 16]
        cache = make_paged(rng, kv_len, 16, 2, 128, torch.bfloat16)
        q = torch.from_numpy(rng.standard_normal((87, 8, 128)).astype(np.float32)).bfloat16().cuda()
        cu, kv = torch.tensor([0, 70, 71, 87], dtype=torch.int32, device="cuda"), torch.tensor(kv_len, dtype=torch.int32, device="cuda")
        lse = torch.zeros(87, 8, device="cuda")
        out = dsp.attend_paged(q, cache, 0, cu, kv, max_new, 0.09, lse=lse)
        check_attend(out, lse, ref_attend(q, cache, 0, new, kv_len, 0.09, True, 0), torch.bfloat16, 200, max_new)


@pytest.mark.parametrize("nH,nKv,hd,dt", [(4, 2, 128, "bf16"), (16, 2, 256, "fp16"), (4, 2, 64, "fp16"), (4, 2, 48, "bf16"), (2, 2, 64, "fp32")])
@pytest.mark.parametrize("new,kv_len", [([3, 150, 2], [3, 400, 40]), ([1, 17], [1, 9000])])
def test_queries_that_are_not_numbers(nH, nKv, hd, dt, new, kv_len):
    """A NaN in a query makes its row NaN and its lse NaN, in one piece or joined from several, and no other row; without
    a key to see, it stays zeros."""
    import block_draft_model_dspark_b200 as dsp
    rng = np.random.default_rng(40)
    dtype, nan = DT[dt], float("nan")
    cache = make_paged(rng, kv_len, 16, nKv, hd, dtype)
    T = sum(new)
    q = torch.from_numpy(rng.standard_normal((T, nH, hd)).astype(np.float32)).to(dtype)
    bad = torch.from_numpy(rng.random((T, nH)) < 0.3)
    bad[T - 1, 0], bad[0, 0] = True, True
    q[bad, int(rng.integers(0, hd))] = nan
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    kv = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    for causal, window in ((True, 0), (False, 0), (True, 33)):
        lse = torch.zeros(T, nH, device="cuda")
        out = dsp.attend_paged(q.cuda(), cache, 0, cu, kv, max(new), hd ** -0.5, causal=causal, window=window, lse=lse).cpu()
        lse = lse.cpu()
        assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
        clean = torch.where(bad[..., None], torch.zeros((), dtype=dtype), q)
        ref = ref_attend(clean, cache, 0, new, kv_len, hd ** -0.5, causal, window)
        zero = torch.where(bad[..., None], ref[0], out.double())
        check_attend(zero, torch.where(bad, ref[2], lse.double()), ref, dtype, max(kv_len), "the other rows")
        assert cache.read_status() == 0


@pytest.mark.parametrize("nH,nKv,hd,dt", [(4, 2, 128, "bf16"), (16, 2, 256, "fp16"), (4, 2, 48, "bf16")])
def test_not_a_number_without_a_key_is_zeros(nH, nKv, hd, dt):
    import block_draft_model_dspark_b200 as dsp
    cache = make_paged(np.random.default_rng(41), [2, 0], 16, nKv, hd, DT[dt])
    q = torch.full((150 + 3, nH, hd), float("nan"), dtype=DT[dt], device="cuda")
    lse = torch.zeros(153, nH, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    out = dsp.attend_paged(q, cache, 0, torch.tensor([0, 150, 153], **i32), torch.tensor([2, 0], **i32), 150, 1.0, lse=lse)
    none = torch.ones(153, dtype=torch.bool)
    none[148:150] = False                                         # the two that sit at keys
    assert bool((out[none.cuda()] == 0).all()) and bool((lse[none.cuda()] == -float("inf")).all())
    assert bool(out[148:150].isnan().all()) and bool(lse[148:150].isnan().all())


@pytest.mark.parametrize("hd,dt", [(128, "bf16"), (256, "fp16"), (48, "fp16")])
def test_one_infinite_score_is_not_a_number(hd, dt):
    """q . K = +infinity for one key alone, whichever column of a tile it is: infinity less infinity. -infinity for all: zeros."""
    import block_draft_model_dspark_b200 as dsp
    i32 = dict(dtype=torch.int32, device="cuda")
    L = 300
    cache = dsp.PagedKvCache(L // 16 + 1, 16, 1, hd, block_table=torch.arange(L // 16 + 1, **i32)[None].contiguous(), dtype=DT[dt])
    q = torch.ones(1, 1, hd, dtype=DT[dt], device="cuda")
    q[:, 0, 3] = float("inf")
    cache.k.view(-1, hd)[:, 3] = -1.0                             # the others: -infinity
    cache.v.fill_(0.5)
    cu, kv = torch.tensor([0, 1], **i32), torch.tensor([L], **i32)
    lse = torch.zeros(1, 1, device="cuda")
    out = dsp.attend_paged(q, cache, 0, cu, kv, 1, 0.1, lse=lse)
    assert bool((out == 0).all()) and float(lse) == -float("inf")
    for j in range(L):
        cache.k.view(-1, hd)[j, 3] = 1.0
        lse = torch.zeros(1, 1, device="cuda")
        out = dsp.attend_paged(q, cache, 0, cu, kv, 1, 0.1, lse=lse)
        assert bool(out.isnan().all()) and bool(lse.isnan().all()), j
        cache.k.view(-1, hd)[j, 3] = -1.0
