"""norm_rope_paged against the formulas in float64: types, head sizes, strides, far positions, padding rows."""
import numpy as np
import pytest
import torch

from paged_util import DT, HALF
from parity_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def ref_heads(x, gain, eps, norm, pos, inv_freq):
    """(y, |a| + |b| of each lane's normed pair) in float64."""
    x = x.double().cpu()
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if gain is not None:
        x = x * gain.double().cpu()
    half = x.shape[-1] // 2
    if inv_freq is None:
        return x, x.abs()
    ang = torch.outer(pos.double().cpu(), inv_freq.double().cpu())[:, None]
    a, b = x[..., :half], x[..., half:]
    y = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    return y, (a.abs() + b.abs()).repeat(1, 1, 2)


def check(got, want, mag, hd, dtype, what):
    # the sum of hd squares, root, division, gain (hd + 8 roundings of 2^-24), the angle (a fraction of a turn
    # rounded to 2^-25, times 2 pi: 2^-22) with its sine and cosine (2^-22), the turn; then the type's rounding
    tol = HALF[dtype] * want.abs() + ((hd + 16) * 2.0 ** -24 + 2.0 ** -21) * mag
    if dtype is torch.float16:
        tol = tol + 2.0 ** -25
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), (what, float((err - tol).max()))


@pytest.mark.parametrize("x,kv", [("fp32", "fp16"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("T,nH,nKv,hd", [(1, 16, 2, 256), (37, 6, 3, 128), (65, 4, 1, 64), (9, 5, 5, 192), (3, 1, 1, 16), (40, 33, 1, 48)])
def test_norm_rope_matches_formula(x, kv, T, nH, nKv, hd):
    import block_draft_model_dspark_b200 as dsp
    g = torch.Generator().manual_seed(T * 100 + hd)
    xt, kt, page = DT[x], DT[kv], 16
    qkv = (torch.randn(T, (nH + 2 * nKv) * hd, generator=g) * 2).to(xt).cuda()        # slices of one product
    q, k, v = (t.unflatten(1, (-1, hd)) for t in qkv.split([nH * hd, nKv * hd, nKv * hd], 1))
    qn, kn = ((1 + 0.2 * torch.randn(hd, generator=g)).to(xt).cuda() for _ in range(2))
    freq = dsp.rope_inv_freq(hd, 1e4, 0.75)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32).cuda()
    pages, layers = T // page + 2, 2
    slots = torch.randperm(pages * page, generator=g)[:T].clone()
    slots[T // 2] = -1 if T > 1 else slots[T // 2]
    slots = slots.cuda()
    for v_norm, layer, vv in ((True, 1, v), (False, 0, v), (True, 0, None)):
        kc, vc = (torch.full((layers, pages, page, nKv, hd), 7.0, dtype=kt, device="cuda") for _ in range(2))
        cache = dsp.PagedKvCache(pages, page, nKv, hd, block_table=torch.zeros(1, 1, dtype=torch.int32, device="cuda"), k=kc, v=vc)
        out = torch.full((T, nH, hd), 5.0, dtype=kt, device="cuda")
        assert dsp.norm_rope_paged(q, k, vv, qn, kn, freq, pos, slots, cache, layer, eps=1e-5, v_norm=v_norm, q_out=out) is out
        real = (slots >= 0).cpu()
        y, mag = ref_heads(q, qn, 1e-5, True, pos, freq)
        check(out[real], y[real], mag[real], hd, kt, "q")
        assert bool((out.cpu()[~real] == 5.0).all())
        at = slots.cpu()[real]
        y, mag = ref_heads(k, kn, 1e-5, True, pos, freq)
        rows = kc[layer].flatten(0, 1).cpu()
        check(rows[at], y[real], mag[real], hd, kt, "k")
        y, mag = ref_heads(v if vv is not None else k, None, 1e-5, v_norm, pos, None)
        vrows = vc[layer].flatten(0, 1).cpu()
        check(vrows[at], y[real], mag[real], hd, kt, "v")
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[at] = False
        for c, rws in ((kc, rows), (vc, vrows)):                      # nothing else is written
            assert bool((rws[rest] == 7.0).all()) and bool((c[1 - layer] == 7.0).all())
        assert cache.read_status() == 0


def test_norm_rope_in_place_and_without_gains():
    import block_draft_model_dspark_b200 as dsp
    g = torch.Generator().manual_seed(3)
    T, nH, hd = 21, 4, 128
    q = torch.randn(T, nH, hd, generator=g).half().cuda()
    k = torch.randn(T, 2, hd, generator=g).half().cuda()
    cache = dsp.PagedKvCache(4, 8, 2, hd, batch=1, max_pages=4, dtype=torch.float16)
    freq, pos = dsp.rope_inv_freq(hd), torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")
    y, mag = ref_heads(q, None, 1e-6, True, pos, freq)
    dsp.norm_rope_paged(q, k, k, None, None, freq, pos, slots, cache, 0, q_out=q)
    check(q, y, mag, hd, torch.float16, "q in place")


def test_norm_rope_slot_past_the_pool_is_skipped():
    import block_draft_model_dspark_b200 as dsp
    cache = dsp.PagedKvCache(2, 8, 1, 64, batch=1, max_pages=2, dtype=torch.bfloat16)
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 9.0)
    dsp.norm_rope_paged(q, k, k, None, None, dsp.rope_inv_freq(64), torch.zeros(3, dtype=torch.int32, device="cuda"),
                        torch.tensor([0, 16, 1 << 40], device="cuda"), cache, 0, q_out=out)
    assert bool((out[1:] == 9.0).all()) and bool((out[0] != 9.0).all())
    assert bool((cache.k.flatten(0, 2)[1:] == 0).all())
    assert cache.read_status() == dsp.DSPARK_DEV_CAPACITY


def test_norm_rope_no_tokens():
    import block_draft_model_dspark_b200 as dsp
    cache = dsp.PagedKvCache(2, 8, 1, 64, batch=1, max_pages=2)
    z = torch.zeros(0, 1, 64, dtype=torch.float16, device="cuda")
    out = dsp.norm_rope_paged(z, z, z, None, None, dsp.rope_inv_freq(64), torch.zeros(0, dtype=torch.int32, device="cuda"),
                              torch.zeros(0, dtype=torch.int64, device="cuda"), cache, 0)
    assert out.shape == (0, 1, 64)


@pytest.mark.parametrize("x,kv", [("bf16", "bf16"), ("fp32", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("T,nH,nKv,hd", [(1200, 32, 8, 128), (1201, 33, 1, 48), (1190, 16, 2, 256), (601, 33, 3, 192), (301, 70, 5, 64), (2400, 7, 7, 16)])
def test_several_rounds_of_heads_a_warp(x, kv, T, nH, nKv, hd):
    """Prompt chunks: a warp has more heads than it takes at a time (one warp per token from 1184 tokens on, several below)."""
    import block_draft_model_dspark_b200 as dsp
    g = torch.Generator().manual_seed(T + hd)
    xt, kt, page = DT[x], DT[kv], 16
    qkv = (torch.randn(T, (nH + 2 * nKv) * hd, generator=g) * 2).to(xt).cuda()
    q, k, v = (t.unflatten(1, (-1, hd)) for t in qkv.split([nH * hd, nKv * hd, nKv * hd], 1))
    qn, kn = ((1 + 0.2 * torch.randn(hd, generator=g)).to(xt).cuda() for _ in range(2))
    freq = dsp.rope_inv_freq(hd, 1e4)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32).cuda()
    pages = T // page + 2
    slots = torch.randperm(pages * page, generator=g)[:T].clone()
    slots[::7] = -1
    for v_norm in (True, False):
        kc, vc = (torch.full((1, pages, page, nKv, hd), 7.0, dtype=kt, device="cuda") for _ in range(2))
        cache = dsp.PagedKvCache(pages, page, nKv, hd, block_table=torch.zeros(1, 1, dtype=torch.int32, device="cuda"), k=kc, v=vc)
        out = torch.full((T, nH, hd), 5.0, dtype=kt, device="cuda")
        dsp.norm_rope_paged(q, k, v, qn, kn, freq, pos, slots.cuda(), cache, 0, eps=1e-5, v_norm=v_norm, q_out=out)
        real, at = slots >= 0, slots[slots >= 0]
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[at] = False
        assert bool((out.cpu()[~real] == 5.0).all())
        y, mag = ref_heads(q, qn, 1e-5, True, pos, freq)
        check(out.cpu()[real], y[real], mag[real], hd, kt, "q")
        for c, src, gain, norm, f, what in ((kc, k, kn, True, freq, "k"), (vc, v, None, v_norm, None, "v")):
            y, mag = ref_heads(src, gain, 1e-5, norm, pos, f)
            rows = c[0].flatten(0, 1).cpu()
            check(rows[at], y[real], mag[real], hd, kt, what)
            assert bool((rows[rest] == 7.0).all())
        assert cache.read_status() == 0
