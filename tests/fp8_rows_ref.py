"""A bound for attention over the 8-bit cache that holds row by row: each query row and
head is measured by what it attends itself, whatever other rows, heads and pages hold."""
from __future__ import annotations

import math

import torch

from paged_ref import ref_attention


def row_bound(x, causal, window=0, scale=None):
    """O and LSE in 64 bits and how far a kernel may be off in each element.

    To ref_attention's errors (products of 16 bits, fp32 sums, one rounding of O) come those
    of a cache of e4m3 c_j times 2^ev_j, for a row with probabilities p_j:
      * A weight is rounded as exp2(s_j + e - m), e being ev_j or at most 3 more, with m at
        least 7 below the row's largest s_j + e: fp16 is off by at most half a step of
        2^-24 at 2^(7 - 3), 2^-29 of the largest p_j 2^ev_j, times |c_j|, over the keys attended.
      * bf16 queries become fp16 times a power of two that puts the row's largest
        element in [2^14, 2^15): an element is off by at most 2^-25, 2^-39 of the largest.
      * s_j + ev_j, the reference and their difference are rounded to fp32 once each:
        three times 2^-24 of |ev_j| more than without it (ref_attention counts those of s_j)."""
    O, L, tol, lse_tol = ref_attention(x, causal, window, scale, least=0.0)
    T, H, d = x.q.shape
    Hkv, page = x.k_cache.shape[1], x.k_cache.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    turned = x.q.dtype is torch.bfloat16
    cu = x.cu.tolist()
    for b, (K, V) in enumerate(zip(x.keys, x.values)):
        t0, t1 = cu[b], cu[b + 1]
        n, Lk = t1 - t0, K.shape[0]
        if n == 0 or Lk == 0:
            continue
        p = torch.arange(n)[:, None] + Lk - n
        j = torch.arange(Lk)[None, :]
        valid = torch.ones(n, Lk, dtype=torch.bool)
        if causal:
            valid &= j <= p
        if window > 0:
            valid &= p - j < window
            if not causal:
                valid &= j - p < window
        cols = torch.arange(Lk) // page
        used = valid.any(0)   # (what no query attends may have any page and scale)
        pages = torch.where(used, x.page_table[b, cols].long(), 0)
        there = used & (pages >= 0) & (pages < x.v_scale.shape[0])
        s = torch.where(there[:, None], x.v_scale[pages.clamp(0, x.v_scale.shape[0] - 1)].double(), 1.0)
        s = torch.where(s == 0, 2.0**-48, s)   # (a page never written to)
        ev = torch.log2(s)                     # [Lk, Hkv]
        for h in range(H):
            hk = h // (H // Hkv)
            q = x.q[t0:t1, h].double()
            S = (q @ K[:, hk].T * scale).masked_fill(~valid, -math.inf)
            z = torch.logsumexp(S, 1)
            lp = S - torch.where(z == -math.inf, 0.0, z)[:, None]
            most = torch.exp((lp + ev[:, hk] * math.log(2)).amax(1))   # largest p_j 2^ev_j
            codes = torch.where(used[:, None], V[:, hk].abs() * torch.exp2(-ev[:, hk])[:, None], 0.0)
            weights = 2.0**-29 * most[:, None] * (valid.double() @ codes)
            e_q = (2.0**-39 * q.abs().amax(1) * scale * (valid.double() * K[:, hk].abs().sum(1)).amax(1)
                   if turned else torch.zeros(n, dtype=torch.float64))
            e_q = e_q + 3 * 2.0**-24 * (valid.double() * ev[:, hk].abs()).amax(1)
            A = torch.exp(lp) @ V[:, hk].abs()
            tol[t0:t1, h] += 2 * e_q[:, None] * A + weights
            lse_tol[h, t0:t1] += e_q
    return O, L, tol, lse_tol


def check_rows(o, lse, x, causal, window=0, scale=None):
    O, L, tol, lse_tol = row_bound(x, causal, window, scale)
    T = int(x.cu[-1])
    o, lse = o.detach().cpu().double()[:T], lse.detach().cpu().double()[:, :T]
    off = (o - O[:T]).abs()
    assert not bool(o.isnan().any()), f"O is NaN in {int(o.isnan().any(2).sum())} rows"
    bad = off > tol[:T]
    assert not bool(bad.any()), (f"{int(bad.sum())} elements of O out of tolerance, up to "
                                 f"{float((off / tol[:T].clamp(min=1e-300)).max()):.3g} times it")
    none = L[:, :T] == -math.inf
    assert torch.equal(none, lse == -math.inf), "rows without a key differ"
    far = torch.where(none, 0.0, lse - L[:, :T]).abs()
    assert bool((far <= lse_tol[:, :T]).all()), f"LSE off by {float(far.nan_to_num(9e9).max()):.3e}"


def rescale_pages(x, b, cols, k_pow=0, v_pow=0, heads=slice(None)):
    """Request b's pages of the given columns times 2^k_pow (keys) and 2^v_pow (values)."""
    page = x.k_cache.shape[2]
    for c in cols:
        pg = int(x.page_table[b, c])
        x.k_scale[pg, heads] *= 2.0**k_pow
        x.v_scale[pg, heads] *= 2.0**v_pow
        x.keys[b][c * page:(c + 1) * page, heads] *= 2.0**k_pow
        x.values[b][c * page:(c + 1) * page, heads] *= 2.0**v_pow
    return x
