"""Plain references of the paged-cache operators in 64 bits (CPU), and the
inputs and tolerances that their tests share."""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch


def ref_page_table(cached, new, table, free_pages, num_free, page_size, max_tokens):
    """cu, seq_lens, slots, pages_taken and the page table after one step, one
    token at a time."""
    table = [list(row) for row in table]
    free = list(free_pages[:num_free])
    cu, seq_lens, slots = [0], [], []
    for b, (c, n) in enumerate(zip(cached, new)):
        for p in range(c, c + n):
            if p % page_size == 0:
                table[b][p // page_size] = free.pop() if free else -1
            page = table[b][p // page_size]
            slots.append(page * page_size + p % page_size if page >= 0 else -1)
        cu.append(cu[-1] + n)
        seq_lens.append(c + n)
    slots += [-1] * (max_tokens - len(slots))
    return cu, seq_lens, slots, num_free - len(free), table


@dataclasses.dataclass
class PagedInputs:
    q: torch.Tensor            # [total_q, H, d]
    k_cache: torch.Tensor      # [num_pages, Hkv, page, d]
    v_cache: torch.Tensor
    page_table: torch.Tensor   # [B, max_pages] int32
    seq_lens: torch.Tensor     # [B] int32
    cu: torch.Tensor           # [B + 1] int32
    max_q: int
    keys: list                 # per request [L, Hkv, d] float64: what the cache holds
    values: list


def make_paged(q_lens, k_lens, H, Hkv, d, page, *, dtype=torch.bfloat16, seed=0, poison=None,
               extra_rows=0, sigma=1.0):
    """Requests with their keys scattered over a shuffled pool.  `poison` fills
    every cache slot that holds no token; unused table entries are -1."""
    g = torch.Generator().manual_seed(seed)
    B, T = len(q_lens), sum(q_lens)
    need = [-(-n // page) for n in k_lens]
    num_pages = sum(need) + 2
    order = torch.randperm(num_pages, generator=g).tolist()
    width = max(1, max(need)) + 1
    table = torch.full((B, width), -1, dtype=torch.int32)
    fill = 0.0 if poison is None else poison
    kc = torch.full((num_pages, Hkv, page, d), fill, dtype=dtype)
    vc = kc.clone()
    keys, values = [], []
    for b, n in enumerate(k_lens):
        k = (torch.randn(n, Hkv, d, generator=g) * sigma).to(dtype)
        v = torch.randn(n, Hkv, d, generator=g).to(dtype)
        keys.append(k.double())
        values.append(v.double())
        for c in range(need[b]):
            pg = order.pop()
            table[b, c] = pg
            m = min(page, n - c * page)
            kc[pg, :, :m] = k[c * page:c * page + m].transpose(0, 1)
            vc[pg, :, :m] = v[c * page:c * page + m].transpose(0, 1)
    q = (torch.randn(T + extra_rows, H, d, generator=g) * sigma).to(dtype)
    cu = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32)
    return PagedInputs(q, kc, vc, table, torch.tensor(k_lens, dtype=torch.int32), cu,
                       max(1, max(q_lens)), keys, values)


def ref_attention(x: PagedInputs, causal, window=0, scale=None, least=None):
    """O, LSE in 64 bits and the largest error that a kernel may have in each
    element, for inputs that are exact in the storage type.  `least`: how far a
    small weight may be off, relative to its row's largest (None: half a step
    below the storage type's normal numbers, over a sum of weights of 1)."""
    T, H, d = x.q.shape
    Hkv = x.k_cache.shape[1]
    dev = x.keys[0].device
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    u = torch.finfo(x.q.dtype).eps / 2
    tiny = torch.finfo(x.q.dtype).smallest_normal * u   # half a step below the normal numbers
    O = torch.zeros(T, H, d, dtype=torch.float64, device=dev)
    tol = torch.zeros(T, H, d, dtype=torch.float64, device=dev)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64, device=dev)
    lse_tol = torch.zeros(H, T, dtype=torch.float64, device=dev)
    cu = x.cu.tolist()
    for b, (K, V) in enumerate(zip(x.keys, x.values)):
        t0, t1 = cu[b], cu[b + 1]
        n, L = t1 - t0, K.shape[0]
        if n == 0 or L == 0:
            continue
        p = torch.arange(n, device=dev)[:, None] + L - n
        j = torch.arange(L, device=dev)[None, :]
        valid = torch.ones(n, L, dtype=torch.bool, device=dev)
        if causal:
            valid &= j <= p
        if window > 0:
            valid &= p - j < window
            if not causal:
                valid &= j - p < window
        for h in range(H):
            q, k, v = x.q[t0:t1, h].double().to(dev), K[:, h // (H // Hkv)], V[:, h // (H // Hkv)]
            S = (q @ k.T * scale).masked_fill(~valid, -math.inf)
            z = torch.logsumexp(S, 1)
            P = torch.exp(S - torch.where(z == -math.inf, 0.0, z)[:, None])
            o, A = P @ v, P @ v.abs()
            # Scores: fp32 sums of d exact products, and one rounding each for
            # the scaled score and its difference from the row's reference;
            # exp2 of the hardware is good to 2^-22.  A weight is then off by
            # e_s relative, and its normaliser by as much again.
            bound = (q.abs() @ k.abs().T * scale).masked_fill(~valid, 0.0).amax(1)
            e_s = (d + 8) * 2.0**-24 * bound + 2.0**-21
            # P rounds to the storage type for the product with V (u), fp32
            # sums over L keys, O rounds once (u).  Below the type's normal
            # numbers (fp16: 2^-14) a rounding is off by up to half a step of
            # the subnormals (2^-25), not by u of the value: of O once, of P for
            # each attended key, whose sum it is divided by is at least 1 (the
            # row's largest weight: a reference never exceeds the maximum).
            below = tiny * (1 + valid.double() @ v.abs())
            if least is not None:   # over the sum of weights relative to the largest
                share = torch.exp(S.amax(1, keepdim=True) - z[:, None]).nan_to_num(0.0)
                below = tiny + least * share * (valid.double() @ v.abs())
            e_o = u + 2 * e_s + (L + 64) * 2.0**-23
            O[t0:t1, h], lse[h, t0:t1] = o, z
            tol[t0:t1, h] = A * (e_o * (1 + u))[:, None] + u * o.abs() + below
            lse_tol[h, t0:t1] = e_s + (L + 64) * 2.0**-24 + z.abs().nan_to_num(0, 0, 0) * 2.0**-22
    return O, lse, tol, lse_tol


def check_attention(o, lse, x: PagedInputs, causal, window=0, scale=None, least=None):
    O, L, tol, lse_tol = ref_attention(x, causal, window, scale, least)
    T = int(x.cu[-1])
    o, lse = o.detach().to(O.device).double(), lse.detach().to(O.device).double()
    over = (o - O).abs()[:T] - tol[:T]
    assert bool((over <= 0).all()), (
        f"O off by {float((o - O).abs()[:T].nan_to_num(9e9).max()):.3e}, "
        f"{int((~(over <= 0)).sum())} of {over.numel()} elements out of tolerance")
    none = L[:, :T] == -math.inf
    assert torch.equal(none, lse[:, :T] == -math.inf), "rows without a key differ"
    d = torch.where(none, 0.0, lse[:, :T] - L[:, :T]).abs() - lse_tol[:, :T]
    assert bool((d <= 0).all()), f"LSE out of tolerance by {float(d.nan_to_num(9e9).max()):.3e}"


# fp16 weights are rounded as multiples of 2^-7 of their row's largest and more:
# the largest is at least 2^7, half a step of the subnormals 2^-25.
FP16_LEAST = 2.0**-32


def put_keys(x: PagedInputs, b, k, v):
    """Gives request b other keys and values ([L, Hkv, d]), in cache and reference."""
    page = x.k_cache.shape[2]
    k, v = k.to(x.q.dtype), v.to(x.q.dtype)
    x.keys[b], x.values[b] = k.double(), v.double()
    for c in range(-(-k.shape[0] // page)):
        m = min(page, k.shape[0] - c * page)
        pg = int(x.page_table[b, c])
        x.k_cache[pg, :, :m] = k[c * page:c * page + m].transpose(0, 1)
        x.v_cache[pg, :, :m] = v[c * page:c * page + m].transpose(0, 1)


def heavy_tail(n, L, heads, d, page, nats, *, every=128, seed=0, dtype=torch.float16):
    """One request in which each `every`-th key outweighs the others by about `nats`
    nats and has the value 0, theirs being 1: O is what the small weights add up
    to, and the bound is relative to that."""
    x = make_paged([n], [L], heads, 1, d, page, dtype=dtype, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    sign = torch.randint(0, 2, (d,), generator=g) * 2.0 - 1.0
    x.q = (sign + 0.02 * torch.randn(n, heads, d, generator=g)).to(dtype)
    k = torch.randn(L, 1, d, generator=g) * 0.7
    k[::every] = sign * (nats / math.sqrt(d))     # q . k / sqrt(d) = nats
    v = torch.ones(L, 1, d)
    v[::every] = 0.0
    put_keys(x, 0, k, v)
    return x


def spread_keys(n, L, H, Hkv, d, page, *, seed=0, dtype=torch.bfloat16):
    """One request whose every 128 keys hold one that some query row gives a large
    share of its weight: with n x H / Hkv rows of a key head and L / 128 such keys
    dealt out to them, losing or misplacing any 128 keys shows in a row."""
    x = make_paged([n], [L], H, Hkv, d, page, dtype=dtype, seed=seed, sigma=0.3)
    g = torch.Generator().manual_seed(seed + 1)
    x.q = torch.randn(n, H, d, generator=g).to(dtype)
    k, v = x.keys[0].clone(), x.values[0].clone()
    G = H // Hkv
    top = math.log(L) + 4     # in sum the other keys weigh e^-4 of one of these
    for j in range(-(-L // 128)):
        at = min(128 * j + int(torch.randint(0, 128, (1,), generator=g)), L - 1)
        row = j % (n * G)
        for hk in range(Hkv):
            q = x.q[row // G, hk * G + row % G].double()
            k[at, hk] = q * (top * math.sqrt(d) / float(q @ q))
    put_keys(x, 0, k, v)
    return x
