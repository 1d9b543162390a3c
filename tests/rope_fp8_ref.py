"""Plain references of rotary positions and of the 8-bit paged cache in 64 bits
(CPU), and the inputs and tolerances that their tests share."""
from __future__ import annotations

import math

import torch

from paged_ref import make_paged, ref_attention

LEAST, MOST, TOP = -48, 48, 448.0


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def ref_rope(x, positions, inv_freq, interleaved=False, inverse=False, scaling=1.0):
    """Rows x [..., d] at integer positions [...]: pair by pair, angles reduced as
    integers times the frequencies' exact values would be (64 bits hold them)."""
    x = x.double()
    half = inv_freq.numel()
    y = x.clone()
    w = positions.double()[..., None] * inv_freq.double()
    c, s = torch.cos(w) * scaling, torch.sin(w) * scaling * (-1 if inverse else 1)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
    return y


def rope_tol(x, ref, positions, inv_freq, interleaved, scaling, dtype):
    """How far a result may be off: cosine and sine by 2^-20 (fp32: 2^-21) and the
    angle by 2^-52 of itself (2^-53 in the kernel's turns, 2^-53 here), two products
    and their sum by 2^-24 each, the result by its type's rounding."""
    half = inv_freq.numel()
    m = x.double().abs()
    eps = (2.0**-21 if dtype is torch.float32 else 2.0**-20) + 4 * 2.0**-24
    eps = eps + (positions.double()[..., None] * inv_freq.double()).abs() * 2.0**-52
    off = torch.zeros_like(m)   # (|a| + |b|) eps of each element's pair
    if interleaved:
        s = (m[..., 0:2 * half:2] + m[..., 1:2 * half:2]) * eps
        off[..., 0:2 * half:2], off[..., 1:2 * half:2] = s, s
    else:
        s = (m[..., :half] + m[..., half:2 * half]) * eps
        off[..., :half], off[..., half:2 * half] = s, s
    off = off * abs(scaling)
    info = torch.finfo(dtype)
    return off * (1 + info.eps) + torch.where(off > 0, ref.abs() * info.eps / 2 + info.smallest_normal * info.eps / 2,
                                              0.0)


# ---------------------------------------------------------------------------
# the 8-bit cache
# ---------------------------------------------------------------------------
def round_e4m3(x):
    """The nearest e4m3 number (ties to even, +-448 at most, NaN stays), 64 bits."""
    part, power = torch.frexp(x)
    normal = torch.ldexp(torch.round(part * 16) / 16, power)
    y = torch.where(x.abs() >= 2.0**-6, normal, torch.round(x * 512) / 512)
    y = torch.where(x.isinf(), torch.sign(x) * TOP, y)
    return y.clamp(-TOP, TOP)


def fit(amax: float) -> int:
    """The smallest exponent in range whose scale holds amax."""
    e = LEAST
    while e < MOST and amax > TOP * 2.0**e:
        e += 1
    return e


def ref_append_fp8(x, cache, exps, slots, page):
    """x [T, Hkv, d], cache [pages, Hkv, page, d] (e4m3 values), exps [pages, Hkv]
    (int), all in 64 bits and changed in place: run by run, head by head."""
    t, T = 0, len(slots)
    while t < T:
        if not 0 <= slots[t] < cache.shape[0] * page:
            t += 1
            continue
        n = 1
        while t + n < T and slots[t + n] == slots[t] + n and slots[t + n] % page:
            n += 1
        p, r = divmod(slots[t], page)
        for h in range(x.shape[1]):
            rows = x[t:t + n, h].double()
            e = fit(float(rows.abs().nan_to_num(0.0, math.inf, math.inf).max()))
            if r > 0:
                old = int(exps[p, h])
                e = max(e, old)
                if e > old:
                    cache[p, h, :r] = round_e4m3(cache[p, h, :r] * 2.0**(old - e))
            exps[p, h] = e
            cache[p, h, r:r + n] = round_e4m3(rows * 2.0**-e)
        t += n


def to_fp8(x, *, spread=0, seed=0, poison=True):
    """PagedInputs with an 8-bit cache: x.k_cache and x.v_cache become e4m3 with
    x.k_scale and x.v_scale, x.keys and x.values what they stand for.  Pages differ in size by
    up to 2^+-spread; slots without a token hold NaN, unused pages' scales are wrong."""
    g = torch.Generator().manual_seed(seed + 77)
    page = x.k_cache.shape[2]
    used = torch.zeros(x.k_cache.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(x.seq_lens.tolist()):
        for c in range(-(-n // page)):
            used[x.page_table[b, c], :min(page, n - c * page)] = True
    for name, cache in (("k", x.k_cache), ("v", x.v_cache)):
        pages, Hkv = cache.shape[:2]
        v = torch.where(used[:, None, :, None], cache.double(), 0.0)
        v = v * torch.exp2(torch.randint(-spread, spread + 1, (pages, Hkv), generator=g).double())[:, :, None, None]
        amax = v.abs().amax((2, 3))
        e = torch.ceil(torch.log2((amax / TOP).clamp(min=1e-14))).clamp(LEAST, MOST)
        codes = round_e4m3(v * torch.exp2(-e)[:, :, None, None])
        scale = torch.exp2(e).float()
        held = codes * torch.exp2(e)[:, :, None, None]
        bits = codes.float().to(torch.float8_e4m3fn).view(torch.uint8)
        if poison:
            bits = torch.where(used[:, None, :, None], bits, 0x7f)
            scale[~used.any(1)] = -3.0
        setattr(x, name + "_cache", bits.view(torch.float8_e4m3fn))
        setattr(x, name + "_scale", scale)
        lists = x.keys if name == "k" else x.values
        for b, n in enumerate(x.seq_lens.tolist()):
            if n:
                ids = x.page_table[b, :-(-n // page)].long()
                lists[b] = held[ids].transpose(1, 2).reshape(-1, Hkv, held.shape[3])[:n].contiguous()
    return x


def make_fp8(*args, spread=0, seed=0, poison=True, **kw):
    return to_fp8(make_paged(*args, seed=seed, **kw), spread=spread, seed=seed, poison=poison)


def check_fp8(o, lse, x, causal, window=0, scale=None):
    """paged_ref's bound for the type of q, whose keys and values are exact in e4m3
    times a power of two.  The kernels multiply in fp16: weights count down to 2^-32 of the
    largest weight times value (kWeightShift), and within a tile of 128 keys e4m3
    values are exact down to 2^-25 of the largest scale."""
    O, L, tol, lse_tol = ref_attention(x, causal, window, scale)
    T, d = int(x.cu[-1]), x.q.shape[2]
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    used = x.page_table[(x.page_table >= 0) & (x.page_table < x.k_cache.shape[0])].long()
    if used.numel():
        k_top, v_top = (float(s[used].nan_to_num(0.0, 0.0, 0.0).max()) for s in (x.k_scale, x.v_scale))
        keys = max(1, int(x.seq_lens.max()))
        e_s = float(x.q[:T].double().abs().sum(2).nan_to_num(0.0).max()) * sc * k_top * 2.0**-25 if T else 0.0
        e_s += 2.0**-38 * float(x.q[:T].double().abs().nan_to_num(0.0).max() if T else 0.0) * d * TOP * k_top * sc
        tol = tol + 2 * e_s * TOP * v_top + keys * TOP * v_top * 2.0**-32
        lse_tol = lse_tol + e_s
    o, lse = o.detach().cpu().double(), lse.detach().cpu().double()
    over = (o - O).abs()[:T] - tol[:T]
    assert bool((over <= 0).all()), (
        f"O off by {float((o - O).abs()[:T].nan_to_num(9e9).max()):.3e}, "
        f"{int((~(over <= 0)).sum())} of {over.numel()} elements out of tolerance")
    none = L[:, :T] == -math.inf
    assert torch.equal(none, lse[:, :T] == -math.inf), "rows without a key differ"
    dl = torch.where(none, 0.0, lse[:, :T] - L[:, :T]).abs() - lse_tol[:, :T]
    assert bool((dl <= 0).all()), f"LSE out of tolerance by {float(dl.nan_to_num(9e9).max()):.3e}"
