"""Inputs and 64-bit references of the paged verification step's operators
(page_slots, norm_rope_paged, attend_paged, sample), shared by their tests.

Tolerances count roundings: HALF[t] is half a step of type t relative to the
value (torch.finfo(t).eps / 2); a 32-bit operation is off by at most 2^-24.
"""
from __future__ import annotations

import math

import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def ceil_div(a: int, b: int) -> int:
    return -(-a // b)


def ref_page_slots(ctx, new, held, free, count, table, page, max_tokens):
    """(n_pages_out, free_count_out, cu, kv, slots, positions, table) by plain loops."""
    table = table.copy()
    B = len(ctx)
    cu, slots, pos, out_pages = [0], [], [], []
    for b in range(B):
        n = list(table[b, :held[b]])
        while len(n) * page < ctx[b] + new[b]:
            count -= 1
            n.append(free[count])
            table[b, len(n) - 1] = n[-1]
        out_pages.append(len(n))
        for i in range(new[b]):
            p = ctx[b] + i
            slots.append(int(n[p // page]) * page + p % page)
            pos.append(p)
        cu.append(cu[-1] + new[b])
    pad = max_tokens - len(slots)
    return (out_pages, count, cu, [c + n for c, n in zip(ctx, new)], slots + [-1] * pad, pos + [0] * pad, table)


def make_paged(rng, kv_len, page, n_kv, hd, dtype, layers=1, extra_pages=2, garbage=True, device="cuda"):
    """A PagedKvCache holding kv_len[b] random rows per request in shuffled pages. Rows that no request
    holds are NaN (garbage=True)."""
    import block_draft_model_dspark_b200 as dsp
    need = [ceil_div(n, page) for n in kv_len]
    pages = sum(need) + extra_pages
    order = rng.permutation(pages)
    table = np.full((len(kv_len), max(need + [1]) + 1), -1, dtype=np.int32)
    shape = (layers, pages, page, n_kv, hd)
    k = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
    v = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
    held = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(kv_len):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for j in range(need[b]):
            held[int(table[b, j]), : min(page, n - j * page)] = True
    if garbage:
        k[:, ~held] = float("nan")
        v[:, ~held] = float("nan")
    cache = dsp.PagedKvCache(pages, page, n_kv, hd, block_table=torch.from_numpy(table).to(device), k=k.to(device), v=v.to(device))
    return cache


def ref_attend(q, cache, layer, new, kv_len, scale, causal, window):
    """Per token: out, sum_j p_j |v_j| / l (what a relative rounding of the p_j can move), lse and the
    largest sum |q_d k_d| (what the scores' rounding scales with), in float64."""
    q = q.double().cpu()
    k, v, table = cache.k[layer].double().cpu(), cache.v[layer].double().cpu(), cache.block_table.cpu().long()
    nH, hd = q.shape[1], q.shape[2]
    grp, T = nH // cache.n_kv, q.shape[0]
    out, mag = torch.zeros(T, nH, hd, dtype=torch.float64), torch.zeros(T, nH, hd, dtype=torch.float64)
    lse = torch.full((T, nH), -math.inf, dtype=torch.float64)
    qk = torch.zeros(T, nH, dtype=torch.float64)
    t0 = 0
    for b, (n, L) in enumerate(zip(new, kv_len)):
        j = torch.arange(L)
        rows = table[b, j // cache.page_size] * cache.page_size + j % cache.page_size
        K, V = k.flatten(0, 1)[rows], v.flatten(0, 1)[rows]
        for i in range(n):
            pos = L - n + i
            see = torch.ones(L, dtype=torch.bool)
            if causal:
                see &= j <= pos
            if window:
                see &= j > pos - window
            if not see.any():
                continue
            Kh, Vh = K[see].repeat_interleave(grp, 1), V[see].repeat_interleave(grp, 1)   # [keys, nH, hd]
            s = torch.einsum("hd,jhd->hj", q[t0 + i], Kh) * scale
            qk[t0 + i] = (torch.einsum("hd,jhd->hj", q[t0 + i].abs(), Kh.abs()) * scale).amax(1)
            lse[t0 + i] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[t0 + i][:, None])
            out[t0 + i] = torch.einsum("hj,jhd->hd", p, Vh)
            mag[t0 + i] = torch.einsum("hj,jhd->hd", p, Vh.abs())
        t0 += n
    return out, mag, lse, qk


def check_attend(got, lse, ref, dtype, keys, what):
    """out: one rounding of each probability and one of the result to `dtype`; the 32-bit sums of `keys`
    terms and of the scores; fp16 probabilities below 2^-14 are off by up to 2^-25 each."""
    out, mag, want_lse, qk = ref
    hd = out.shape[2]
    h = HALF[dtype]
    score = (hd + 4) * 2.0 ** -24 * qk                         # error of a score, absolute; of a probability, relative
    tol = h * (out.abs() + mag) + (2 * score[..., None] + (keys + 64) * 2.0 ** -23) * mag + 1e-30
    if dtype is torch.float16:
        tol = tol + keys * 2.0 ** -25 * 8 + 2.0 ** -24
    err = (got.double().cpu() - out).abs()
    assert bool((err <= tol).all()), (what, float((err - tol).max()), float(err.max()))
    if lse is not None:
        lse = lse.double().cpu()
        none = want_lse == -math.inf
        assert bool((lse[none] == -math.inf).all()), what
        e = (lse - want_lse).abs()[~none]
        t = (score + (keys + 64) * 2.0 ** -23 + want_lse.abs() * 2.0 ** -22)[~none]
        assert bool((e <= t).all()), (what, "lse", float((e - t).max()))


def ref_sample(x, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(token, share, margin) per row in float64; margin: the distance of u * total from the nearest edge of the
    drawn token, and of every mass edge that decided a filter, relative to the total."""
    R, V = x.shape
    tok, prob, margin = np.empty(R, np.int64), np.empty(R), np.empty(R)
    for r in range(R):
        z = np.where(np.isnan(x[r]), -np.inf, x[r].astype(np.float64)) + 0.0
        m = z.max()
        T = 1.0 if temperature is None else float(temperature[r])
        if m == -np.inf:
            tok[r], prob[r], margin[r] = -1, 0.0, 1.0
            continue
        if not T > 0:
            tok[r], prob[r], margin[r] = int(np.argmax(z)), 1.0, 1.0
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            w = np.where(z == m, 1.0, np.exp((z - m) / T))
        order = np.argsort(-z, kind="stable")
        keep, near = order, 1.0
        if top_k is not None and top_k[r] > 0:
            keep = keep[: int(top_k[r])]
        if top_p is not None and top_p[r] < 1:
            c = np.cumsum(w[keep])
            edge = float(top_p[r]) * c[-1]
            n = max(1, int(np.count_nonzero(c - w[keep] < edge)))
            near = min(near, np.abs(c - w[keep] - edge).min() / c[-1]) if top_p[r] > 0 else near
            keep = keep[:n]
        if min_p is not None and min_p[r] > 0:
            k0 = keep[0]
            keep = keep[(w[keep] >= float(min_p[r])) | (keep == k0)]
        keep = np.sort(keep)
        c = np.cumsum(w[keep])
        want = float(u[r]) * c[-1]
        i = min(int(np.count_nonzero(c <= want)), len(keep) - 1)
        near = min(near, np.abs(np.concatenate([c[:-1], [np.inf]]) - want).min() / c[-1])
        tok[r], prob[r], margin[r] = keep[i], w[keep[i]] / c[-1], near
    return tok, prob, margin
