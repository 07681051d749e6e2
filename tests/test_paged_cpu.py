"""The paged verification step's C entry points without a GPU: every refusal returns its code, with a message,
before anything is launched (the pointers here are numbers that nothing may touch)."""
import ctypes
import os
import re

import numpy as np
import pytest

P = 4096            # an aligned address that is never read


@pytest.fixture(scope="module")
def dsp():
    from block_draft_model_dspark_b200 import build
    build.build()
    import block_draft_model_dspark_b200 as d
    d.get_lib()
    return d


def cache(dsp, **kw):
    c = dsp.dspark_paged_cache()
    c.k = c.v = c.block_table = P
    c.layers, c.num_pages, c.page_size, c.n_kv, c.head_dim, c.batch, c.max_pages, c.dtype = 2, 10, 16, 2, 128, 8, 4, dsp.DSPARK_DTYPE_F16
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def refused(dsp, rc, code):
    assert rc == code and dsp.get_lib().dspark_last_error().decode()


BAD_CACHES = [(dict(layers=0), -1), (dict(num_pages=0), -1), (dict(page_size=0), -1), (dict(n_kv=0), -1), (dict(batch=0), -1), (dict(max_pages=0), -1),
              (dict(dtype=3), -1), (dict(head_dim=0), -2), (dict(head_dim=100), -2), (dict(head_dim=512), -2), (dict(block_table=None), -1),
              (dict(page_size=1 << 21), -2), (dict(n_kv=1 << 17), -2)]


def slots_args(c, **kw):
    a = dict(cache=ctypes.addressof(c), ctx_len=P, n_new=P, B=8, n_pages=P, free_pages=P, n_free=4, free_count=P, max_tokens=5, n_pages_out=P,
             free_count_out=P, cu_new=P, kv_len=P, slots=P, positions=P, stream=None)
    a.update(kw)
    return list(a.values())


def norm_args(c, **kw):
    a = dict(cache=ctypes.addressof(c), layer=1, x_dtype=1, q=P, q_stride=1024, k=P, k_stride=1024, v=P, v_stride=1024, n_heads=4, q_norm=P, k_norm=P,
             inv_freq=P, eps=1e-6, v_norm=0, positions=P, slots=P, T=3, q_out=P, stream=None)
    a.update(kw)
    return list(a.values())


def attend_args(c, **kw):
    a = dict(cache=ctypes.addressof(c), layer=1, q=P, q_stride=512, n_heads=4, cu_new=P, kv_len=P, B=8, T=3, max_new=2, scale=0.1, causal=1, window=0,
             out=P, out_stride=512, lse=None, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return list(a.values())


def sample_args(**kw):
    a = dict(logits=P, dtype=0, row_stride=100, rows=2, vocab=100, u=P, temperature=None, top_k=None, top_p=None, min_p=None, tokens=P, probs=None, ws=P,
             ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(dsp, kw, code):
    lib, c = dsp.get_lib(), cache(dsp, **kw)
    refused(dsp, lib.dspark_page_slots(*slots_args(c)), code)
    refused(dsp, lib.dspark_norm_rope_paged(*norm_args(c)), code)
    refused(dsp, lib.dspark_attend_paged(*attend_args(c)), code)
    assert lib.dspark_attend_paged_workspace_bytes(ctypes.addressof(c), 10, 4, 8) == 0


def test_page_slots_refusals(dsp):
    lib, c = dsp.get_lib(), cache(dsp)
    refused(dsp, lib.dspark_page_slots(*slots_args(c, cache=None)), -1)
    for kw in (dict(B=0), dict(B=9), dict(max_tokens=-1), dict(n_free=-1)) + tuple({n: None} for n in
               ("ctx_len", "n_new", "n_pages", "free_pages", "free_count", "n_pages_out", "free_count_out", "cu_new", "kv_len", "slots", "positions")):
        refused(dsp, lib.dspark_page_slots(*slots_args(c, **kw)), -1)
    big = cache(dsp, batch=5000)
    refused(dsp, lib.dspark_page_slots(*slots_args(big, B=4097)), -2)
    refused(dsp, lib.dspark_page_slots(*slots_args(c, max_tokens=(1 << 30) + 1)), -2)


def test_norm_rope_refusals(dsp):
    lib, c = dsp.get_lib(), cache(dsp)
    for kw in (dict(layer=-1), dict(layer=2), dict(x_dtype=7), dict(n_heads=0), dict(T=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(q=P + 8), dict(k=P + 2),
               dict(v=P + 8), dict(q_out=P + 8), dict(q_norm=P + 8), dict(k_norm=P + 4), dict(q_stride=1001), dict(k_stride=4), dict(v_stride=2)) + \
            tuple({n: None} for n in ("q", "k", "inv_freq", "positions", "slots", "q_out")):
        refused(dsp, lib.dspark_norm_rope_paged(*norm_args(c, **kw)), -1)
    for kw in (dict(k=None), dict(v=None), dict(k=P + 8)):
        bad = cache(dsp, **kw)
        refused(dsp, lib.dspark_norm_rope_paged(*norm_args(bad)), -1)
    assert lib.dspark_norm_rope_paged(*norm_args(c, T=0, q=None, k=None)) == 0


def test_attend_refusals(dsp):
    lib, c = dsp.get_lib(), cache(dsp)
    for kw in (dict(layer=-1), dict(layer=2), dict(n_heads=0), dict(n_heads=3), dict(B=-1), dict(B=9), dict(T=-1), dict(max_new=-1), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(q=P + 8), dict(out=P + 8), dict(ws=P + 16),
               dict(q_stride=100), dict(out_stride=100), dict(q_stride=-512), dict(out_stride=-512)) + tuple({n: None} for n in ("q", "out", "cu_new", "kv_len", "ws")):
        refused(dsp, lib.dspark_attend_paged(*attend_args(c, **kw)), -1)
    for kw in (dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 8)):
        bad = cache(dsp, **kw)
        refused(dsp, lib.dspark_attend_paged(*attend_args(bad)), -1)
    need = lib.dspark_attend_paged_workspace_bytes(ctypes.addressof(c), 3, 4, 8)
    assert need > 0
    refused(dsp, lib.dspark_attend_paged(*attend_args(c, ws_bytes=need - 1)), -4)
    refused(dsp, lib.dspark_attend_paged(*attend_args(c, T=1 << 30)), -2)
    for kw in (dict(q_stride=504), dict(out_stride=256)):           # tokens that overlap
        refused(dsp, lib.dspark_attend_paged(*attend_args(c, **kw)), -1)
    big = cache(dsp, batch=5000)
    refused(dsp, lib.dspark_attend_paged(*attend_args(big, B=4097)), -2)
    assert lib.dspark_attend_paged(*attend_args(c, T=0, q=None)) == 0
    assert lib.dspark_attend_paged(*attend_args(c, B=0, kv_len=None)) == 0


def test_sample_refusals(dsp):
    lib = dsp.get_lib()
    for kw in (dict(dtype=5), dict(rows=-1), dict(vocab=0), dict(row_stride=99), dict(logits=None), dict(u=None), dict(tokens=None), dict(ws=None),
               dict(logits=P + 2), dict(ws=P + 16)):
        refused(dsp, lib.dspark_sample(*sample_args(**kw)), -1)
    refused(dsp, lib.dspark_sample(*sample_args(vocab=(1 << 24) + 1, row_stride=1 << 25)), -2)
    need = lib.dspark_sample_workspace_bytes(2, 100)
    assert need > 0 and lib.dspark_sample_workspace_bytes(-1, 100) == 0 and lib.dspark_sample_workspace_bytes(1, 0) == 0
    refused(dsp, lib.dspark_sample(*sample_args(ws_bytes=need - 1)), -4)
    assert lib.dspark_sample(*sample_args(rows=0, logits=None)) == 0


def test_packed_calls_refuse_alike(dsp):
    """The same call as a block of 64-bit words: the same result and message, argument by argument."""
    import struct
    lib, c = dsp.get_lib(), cache(dsp)

    def both(call, plain, args):
        words = struct.pack("@" + "".join("d" if isinstance(a, float) else "q" for a in args), *[0 if a is None else a for a in args])
        want, msg = plain(*args), dsp.get_lib().dspark_last_error()
        assert lib.dspark_packed_call(call, words) == want and dsp.get_lib().dspark_last_error() == msg
        return want

    for kw in (dict(B=9), dict(free_pages=None), dict(max_tokens=-1), dict(positions=None)):
        assert both(0, lib.dspark_page_slots, slots_args(c, **kw)) == -1
    for kw in (dict(layer=2), dict(x_dtype=7), dict(eps=-1.0), dict(k_stride=4), dict(q_out=None), dict(T=-1)):
        assert both(1, lib.dspark_norm_rope_paged, norm_args(c, **kw)) == -1
    assert both(1, lib.dspark_norm_rope_paged, norm_args(c, T=0)) == 0
    for kw in (dict(scale=0.0), dict(window=-1), dict(B=9), dict(out_stride=100), dict(ws=None)):
        assert both(2, lib.dspark_attend_paged, attend_args(c, **kw)) == -1
    assert both(2, lib.dspark_attend_paged, attend_args(c, ws_bytes=8)) == -4
    for kw in (dict(dtype=5), dict(row_stride=99), dict(tokens=None), dict(ws=P + 16)):
        assert both(3, lib.dspark_sample, sample_args(**kw)) == -1
    assert both(3, lib.dspark_sample, sample_args(rows=0)) == 0
    refused(dsp, lib.dspark_packed_call(4, b"\0" * 160), -1)
    refused(dsp, lib.dspark_packed_call(0, None), -1)


def test_packed_integers_past_32_bits_are_refused(dsp):
    """Not cut to their low half. Each call has another fault too (a NULL, a scale of 0), so that none could ever launch."""
    import struct
    lib, c = dsp.get_lib(), cache(dsp)
    calls = [(0, slots_args(c, slots=None), (3, 6, 8)), (1, norm_args(c, q_out=None), (1, 2, 9, 14, 17)),
             (2, attend_args(c, scale=0.0), (1, 4, 7, 8, 9, 11, 12)), (3, sample_args(tokens=None), (1, 3, 4))]
    for call, args, where in calls:
        for i in where:
            for far in (1 << 32, -(1 << 32), 1 << 31, 1 << 62):
                bad = [0 if a is None else a for a in args]
                bad[i] += far
                words = struct.pack("@" + "".join("d" if isinstance(a, float) else "q" for a in bad), *bad)
                refused(dsp, lib.dspark_packed_call(call, words), -1)
                assert b"32 bits" in lib.dspark_last_error(), (call, i, far, lib.dspark_last_error())


def test_attention_polynomial_is_as_close_as_its_comment_says():
    """2^f on |f| <= 1/2 by the kernel's coefficients, in fp32 with fused multiply-adds: within 2^-22."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "block_draft_model_dspark_b200", "csrc", "attend_paged_tc.cu")) as f:
        body = re.search(r"void exp2_poly\(.*?\n}", f.read(), re.S).group(0)
    pair = r"f2\(([\d.e-]+)f, \1f\)"
    first = re.search(r"fma2\(" + pair + r", f, " + pair.replace("\\1", "\\2") + r"\)", body)
    rest = re.findall(r"p = fma2\(p, f, " + pair + r"\)", body)
    c = [np.float32(v) for v in list(first.groups()) + rest]
    assert len(c) == 6
    x = np.linspace(-0.5, 0.5, 1 << 20).astype(np.float32)
    p = np.full_like(x, c[0])
    for k in c[1:]:                                       # a product of two fp32 is exact in 64 bits, the sum far more exact than fp32
        p = (p.astype(np.float64) * x.astype(np.float64) + np.float64(k)).astype(np.float32)
    t = np.exp2(x.astype(np.float64))
    assert np.abs(p.astype(np.float64) / t - 1).max() < 2.0 ** -22
