"""Rotary positions and the paged cache held in 8 bits, as workloads to time.

Four operators: ``attn_rope`` (rotary positions of queries and keys, and the
gradient), ``attn_cache_append_rope`` (a step's queries and keys rotated, keys
and values written to their slots), ``attn_cache_append_fp8`` (keys and values
rounded to e4m3 with one scale per page and head) and ``attn_fwd_paged_fp8``
(attention of new tokens over such a cache).  ``run`` computes them in plain
torch operations, or through the package where ``own`` is true.  A case holds
plain values; its request lengths come from its own ``lens_seed``, the tensors'
values and the page order from the seed given to ``prepare``.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_LEAST, _MOST = -48, 48   # exponents of a cache's scales
_TOP = 448.0              # largest e4m3 number


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rope(name, B, H, Hk, N, d, r, dtype="bf16", interleaved=False, inverse=False, packed=False,
          far=0, base=10000.0, scaling=1.0):
    return {"name": name, "op": "rope", "B": B, "H": H, "Hk": Hk, "N": N, "d": d, "r": r,
            "dtype": dtype, "interleaved": interleaved, "inverse": inverse, "packed": packed,
            "far": far, "base": base, "scaling": scaling}


def _step(op, name, B, q, ctx, Hq, Hkv, d, page, dtype, lens_seed, **more):
    return {"name": name, "op": op, "B": B, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype,
            "lens_seed": lens_seed, **more}


def _append_rope(name, B, q, ctx, Hq, Hkv, d, page, r, dtype="bf16", interleaved=False,
                 base=10000.0, scaling=1.0, lens_seed=1):
    return _step("append_rope", name, B, q, ctx, Hq, Hkv, d, page, dtype, lens_seed, r=r,
                 interleaved=interleaved, base=base, scaling=scaling)


def _append8(name, B, q, ctx, Hkv, d, page, dtype="bf16", lens_seed=1):
    return _step("append8", name, B, q, ctx, Hkv, Hkv, d, page, dtype, lens_seed)


def _attend8(name, B, q, ctx, Hq, Hkv, d, page, dtype="bf16", causal=True, window=0, lens_seed=1):
    return _step("attend8", name, B, q, ctx, Hq, Hkv, d, page, dtype, lens_seed, causal=causal,
                 window=window)


def listed():
    return [
        # The queries and keys of one decoding step of 48 requests far into
        # their contexts, positions as a tensor: latency.
        _rope("rope_token_t48_h32k8_d128", 1, 32, 8, 48, 128, 128, packed=True, far=131072,
              base=500000.0),
        # Queries and keys of a training step at the 4 x 16 x 4096 x 128 shape.
        _rope("rope_train_b4_h16_n4096_d128", 4, 16, 16, 4096, 128, 128),
        # The gradient at the 8 x 12 x 1024 x 64 shape: interleaved pairs, half
        # of the head, a factor for long contexts.
        _rope("rope_grad_b8_h12_n1024_d64", 8, 12, 12, 1024, 64, 32, dtype="fp16",
              interleaved=True, inverse=True, scaling=1.1386),
        # One decoding step, and one step of prompt chunks, into a 16-bit cache.
        _append_rope("append_rope_token_b64", 64, (1, 1), (100, 5000), 32, 8, 128, 16, 128),
        _append_rope("append_rope_prompt_b16", 16, (900, 1100), (0, 1000), 16, 4, 128, 64, 64,
                     dtype="fp16", interleaved=True, lens_seed=2),
        # The same two steps into a cache of 8 bits.
        _append8("append8_token_b64", 64, (1, 1), (100, 5000), 8, 128, 16),
        _append8("append8_prompt_b16", 16, (900, 1100), (0, 1000), 8, 128, 64, lens_seed=2),
        # One interactive request of a 12-head, d = 64 model: latency.
        _attend8("token8_b1_h12_d64", 1, (1, 1), (997, 997), 12, 12, 64, 16),
        # A serving batch, one token per request, ragged contexts: bound by
        # reading the cache.
        _attend8("token8_b48_h32kv8_d128", 48, (1, 1), (130, 4200), 32, 8, 128, 16, lens_seed=2),
        # Two very long contexts with few key heads.
        _attend8("token8_long_b2_h16kv2_d128", 2, (1, 1), (70001, 131072), 16, 2, 128, 64,
                 lens_seed=3),
        # A chunk of a long prompt over what is already cached.
        _attend8("chunk8_b1_h16_d128", 1, (512, 512), (16100, 16100), 16, 16, 128, 64),
        # A mixed step: prompt chunks beside single tokens, sliding window, odd
        # page size, fp16.
        _attend8("mixed8_b12_h16kv4_d64_window", 12, (1, 700), (0, 3500), 16, 4, 64, 48,
                 dtype="fp16", window=1024, lens_seed=6),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "append_rope", "append8", "attend8", "attend8", "attend8"])
    seed = rng.randrange(1 << 30)
    page = rng.choice([8, 16, 16, 32, 48, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    d = rng.choice([64, 128, 128, 256])
    r = rng.choice([d, d, d // 2, d // 4, rng.randrange(16, d + 1, 16)])
    base = rng.choice([10000.0, 500000.0])
    scaling = rng.choice([1.0, 1.0, 1.2])
    if op == "rope":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        packed = rng.random() < 0.5
        Hk, G = rng.choice([1, 2, 4, 8, 12, 16]), rng.choice([1, 2, 4, 7])
        if packed:
            B, N = 1, _log_int(rng, 1, 8000)
        else:
            B, N = _log_int(rng, 1, 8), _log_int(rng, 1, 4096)
        while G > 1 and Hk * G > 32:
            G -= 1
        while B > 1 and B * N * Hk * (G + 1) * d > 4 * 2 * 16 * 4096 * 128:
            B -= 1
        while N > 1 and B * N * Hk * (G + 1) * d > 4 * 2 * 16 * 4096 * 128:
            N = N * 2 // 3
        if dtype == "fp32":
            N = max(1, N // 2)
        case = _rope(None, B, Hk * G, Hk, N, d, r, dtype, rng.random() < 0.5, rng.random() < 0.5,
                     packed, _log_int(rng, 1000, 1000000) if packed else 0, base, scaling)
    elif op in ("append_rope", "append8"):
        q_hi = rng.choice([1, _log_int(rng, 2, 1100)])
        B = _log_int(rng, 1, 64 if q_hi < 250 else 16)
        ctx = (0, _log_int(rng, 10, 5000))
        Hkv, d = rng.choice([1, 2, 4, 8]), min(d, 128)
        if op == "append8":
            case = _append8(None, B, (1, q_hi), ctx, Hkv, d, page, dtype, seed)
        else:
            case = _append_rope(None, B, (1, q_hi), ctx, Hkv * rng.choice([1, 2, 4]), Hkv, d, page,
                                min(r, d), dtype, rng.random() < 0.5, base, scaling, seed)
    else:
        Hkv = rng.choice([1, 2, 4, 8, 12, 16])
        G = rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
        kind = rng.choice(["token", "token", "verify", "chunk", "prompt"])
        causal, window = True, rng.choice([0, 0, 0, _log_int(rng, 20, 2000)])
        if kind == "token":
            q, ctx_hi, B = (1, 1), _log_int(rng, 50, 130000), _log_int(rng, 1, 48)
        elif kind == "verify":
            q_hi = rng.randrange(2, 9)
            q, ctx_hi, B = (q_hi, q_hi), _log_int(rng, 50, 20000), _log_int(rng, 1, 32)
        elif kind == "chunk":
            q_hi = _log_int(rng, 16, 700)
            q, ctx_hi, B = (1, q_hi), _log_int(rng, 50, 16000), _log_int(rng, 1, 12)
            causal = rng.random() < 0.8
        else:
            q_hi = _log_int(rng, 100, 2048)
            q, ctx_hi, B = (max(1, q_hi // 2), q_hi), 1, _log_int(rng, 1, 8)
        while G > 1 and Hkv * G > 32:
            G -= 1
        # no more products than the chunk of 512 over 16100 keys, and no more
        # cached elements than 48 requests of up to 4200 tokens, 8 heads, d = 128
        while B > 1 and (B * Hkv * G * q[1] * (q[1] + ctx_hi) * d > 16 * 512 * 16612 * 128
                         or B * Hkv * (q[1] + ctx_hi) * d > 30 * 4200 * 8 * 128):
            B -= 1
        while Hkv > 1 and (Hkv * (q[1] + ctx_hi) * d > 24 * 4200 * 8 * 128
                           or Hkv * G * q[1] * (q[1] + ctx_hi) * d > 16 * 512 * 16612 * 128):
            Hkv //= 2
        case = _attend8(None, B, q, (ctx_hi // 3, ctx_hi), Hkv * G, Hkv, d, page, dtype, causal,
                        window, seed)
    del case["name"]
    return case


def _lengths(case):
    """New tokens and cached tokens of every request."""
    rng = random.Random(case["lens_seed"])
    new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    cached = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    return new, cached


def _pages(n, page):
    return -(-n // page)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _exponent(amax):
    """The smallest e with amax <= 448 2^e, within the scales' range."""
    m, x = torch.frexp(amax.float())   # amax = m 2^x, m in [0.5, 1); 448 = 0.875 2^9
    e = (x - 9 + (m > 0.875).to(torch.int32)).clamp(_LEAST, _MOST)
    return torch.where(amax > 0, e, _LEAST)


def _power(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def _round8(x, scale):
    return (x.float() / scale).clamp(-_TOP, _TOP).to(torch.float8_e4m3fn)


def _quantise(x):
    """[pages, heads, rows, d] -> e4m3 and the scale of each page and head."""
    s = _power(_exponent(x.float().abs().amax((2, 3))))
    return _round8(x, s[:, :, None, None]), s


def _inv_freq(case):
    i = torch.arange(0, case["r"], 2, dtype=torch.float64, device="cuda")
    return (case["base"] ** (-i / case["r"])).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).to(dtype)

    if case["op"] == "rope":
        B, N, d = case["B"], case["N"], case["d"]
        s = {k: case[k] for k in ("op", "interleaved", "inverse", "scaling")}
        s["inv_freq"], s["positions"] = _inv_freq(case), None
        if case["packed"]:
            s["q"], s["k"] = randn(N, case["H"], d), randn(N, case["Hk"], d)
            s["positions"] = torch.randint(0, case["far"], (N,), device="cuda", generator=gen,
                                           dtype=torch.int32)
        else:
            s["q"], s["k"] = randn(B, case["H"], N, d), randn(B, case["Hk"], N, d)
        return s

    new, cached = _lengths(case)
    lens = [n + c for n, c in zip(new, cached)]
    page, B, T = case["page"], case["B"], sum(new)
    Hkv, d = case["Hkv"], case["d"]

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    # Pages in the order in which a busy pool hands them out: any.
    filled = [_pages(x, page) for x in lens]
    num_pages = sum(filled) + max(2, sum(filled) // 8)
    order = torch.randperm(num_pages, device="cuda", generator=gen).to(torch.int32)
    starts = torch.tensor([0] + filled[:-1], device="cuda").cumsum(0)
    col = torch.arange(max(filled), device="cuda")
    table = torch.where(col < torch.tensor(filled, device="cuda")[:, None],
                        order[(starts[:, None] + col).clamp(max=num_pages - 1)],
                        -1).to(torch.int32).contiguous()
    cu = i32([0] + new).cumsum(0).to(torch.int32)
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(new, device="cuda"))
    pos = torch.arange(T, device="cuda") - cu.long()[b] + i32(cached).long()[b]
    s = {"op": case["op"], "page": page, "cu": cu, "seq_lens": i32(lens),
         "slots": table[b, pos // page].long() * page + pos % page}
    if case["op"] == "append_rope":
        s.update(q=randn(T, case["Hq"], d), k=randn(T, Hkv, d), v=randn(T, Hkv, d),
                 k_cache=randn(num_pages, Hkv, page, d), v_cache=randn(num_pages, Hkv, page, d),
                 inv_freq=_inv_freq(case), interleaved=case["interleaved"],
                 scaling=case["scaling"])
        return s

    # Keys and values of 8 bits: channels of unlike size, as trained models have
    # them, so that the pages' scales differ.
    width = torch.exp(torch.randn(2, Hkv, 1, d, device="cuda", generator=gen) * 0.5)
    s["k_cache"], s["k_scale"] = _quantise(randn(num_pages, Hkv, page, d) * width[0])
    s["v_cache"], s["v_scale"] = _quantise(randn(num_pages, Hkv, page, d) * width[1])
    if case["op"] == "append8":
        s["k"] = (randn(T, Hkv, d) * width[0, :, 0]).to(dtype)
        s["v"] = (randn(T, Hkv, d) * width[1, :, 0]).to(dtype)
        return s
    s.update(q=randn(T, case["Hq"], d), table=table, max_q=max(new), max_k=max(lens),
             causal=case["causal"], window=case["window"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return {"rope": _run_rope, "append_rope": _run_append_rope, "append8": _run_append8,
            "attend8": _run_attend8}[state["op"]](state)


def _rotate(x, positions, inv_freq, interleaved, inverse, scaling):
    """x [..., d] rotated by positions [...] (of x's leading shape or less): the
    angles in 64 bits, where far positions need them."""
    angle = positions.double()[..., None] * inv_freq.double()
    cos, sin = (angle.cos() * scaling).float(), (angle.sin() * scaling).float()
    if inverse:
        sin = -sin
    half = inv_freq.numel()
    r = 2 * half
    y = x.float()
    if interleaved:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        z = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:r]
        z = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((z, y[..., r:]), -1).to(x.dtype)


def _run_rope(s):
    if own:
        import exact_attention_58_gb300 as ea
        return ea.attn_rope(s["q"], s["k"], s["inv_freq"], s["positions"],
                            interleaved=s["interleaved"], inverse=s["inverse"],
                            scaling=s["scaling"])
    if s["positions"] is None:
        pos = torch.arange(s["q"].shape[2], device=s["q"].device)
    else:
        pos = s["positions"][:, None]
    return tuple(_rotate(x, pos, s["inv_freq"], s["interleaved"], s["inverse"], s["scaling"])
                 for x in (s["q"], s["k"]))


def _request_of(cu, T):
    t = torch.arange(T, device=cu.device)
    return t, torch.searchsorted(cu[1:].contiguous(), t, right=True)


def _run_append_rope(s):
    if own:
        import exact_attention_58_gb300 as ea
        q = ea.attn_cache_append_rope(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                      s["slots"], s["inv_freq"], cu_seqlens_q=s["cu"],
                                      seq_lens=s["seq_lens"], interleaved=s["interleaved"],
                                      scaling=s["scaling"])
        return q, s["k_cache"], s["v_cache"]
    cu = s["cu"].long()
    t, b = _request_of(cu, s["q"].shape[0])
    pos = (s["seq_lens"].long()[b] - cu[b + 1] + t)[:, None]
    rope = (s["inv_freq"], s["interleaved"], False, s["scaling"])
    page, row = s["slots"] // s["page"], s["slots"] % s["page"]
    s["k_cache"][page, :, row] = _rotate(s["k"], pos, *rope)
    s["v_cache"][page, :, row] = s["v"]
    return _rotate(s["q"], pos, *rope), s["k_cache"], s["v_cache"]


def _run_append8(s):
    if own:
        import exact_attention_58_gb300 as ea
        ea.attn_cache_append_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"],
                                 s["v_scale"], s["slots"])
    else:
        _append8_plain(s["k"], s["k_cache"], s["k_scale"], s["slots"])
        _append8_plain(s["v"], s["v_cache"], s["v_scale"], s["slots"])
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _append8_plain(x, cache, scale, slots):
    pages, _, size, d = cache.shape
    page, row = slots // size, slots % size
    Hkv = x.shape[1]
    # the first row written in each page (its size where none is)
    first = torch.full((pages,), size, device=x.device).scatter_reduce_(0, page, row, "amin")
    amax = torch.zeros(pages, Hkv, device=x.device).scatter_reduce_(
        0, page[:, None].expand(-1, Hkv), x.float().abs().amax(2), "amax")
    old = torch.where((first > 0)[:, None], _exponent(scale * _TOP), _LEAST)
    e = torch.maximum(_exponent(amax), old)
    grown = _power(e)
    # rows that the page held already, on the new scale
    ids = torch.unique(page)
    held = cache[ids].float() * scale[ids][:, :, None, None]
    keep = torch.arange(size, device=x.device)[None, :] < first[ids, None]
    again = _round8(held, grown[ids][:, :, None, None]).view(torch.uint8)
    bits = cache.view(torch.uint8)
    bits[ids] = torch.where(keep[:, None, :, None], again, bits[ids])
    bits[page, :, row] = _round8(x, grown[page][:, :, None]).view(torch.uint8)
    scale[ids] = grown[ids]


def _run_attend8(s):
    if own:
        import exact_attention_58_gb300 as ea
        return ea.attn_fwd_paged_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"],
                                     s["v_scale"], s["table"], s["seq_lens"], s["cu"], s["max_q"],
                                     causal=s["causal"], window=s["window"])
    q, cu, seq_lens = s["q"], s["cu"].long(), s["seq_lens"].long()
    T, Hq, d = q.shape
    _, Hkv, page, _ = s["k_cache"].shape
    B, G, dev = cu.numel() - 1, Hq // Hkv, q.device
    ids = s["table"][:, :_pages(s["max_k"], page)].clamp(min=0).long()

    def keys(cache, scale):   # [B, Hkv, keys, d]
        x = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
        return (x * scale[ids][..., None, None]).transpose(1, 2).reshape(B, Hkv, -1, d)

    k, v = keys(s["k_cache"], s["k_scale"]), keys(s["v_cache"], s["v_scale"])
    # the queries of every request, padded to the longest: [B, Hkv, max_q * G, d]
    i = torch.arange(s["max_q"], device=dev)
    rows = (cu[:-1, None] + i).clamp(max=T - 1)
    qp = q[rows].float().reshape(B, -1, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, -1, d)
    scores = (qp @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).reshape(B, Hkv, -1, G, k.shape[2])
    # query i stands at key position i + (keys - queries)
    j = torch.arange(k.shape[2], device=dev)
    p = (i + (seq_lens - cu[1:] + cu[:-1])[:, None])[:, :, None]
    valid = (j < seq_lens[:, None, None]).expand(B, i.numel(), j.numel())
    if s["causal"]:
        valid = valid & (j <= p)
    if s["window"] > 0:
        valid = valid & (p - j < s["window"])
        if not s["causal"]:
            valid = valid & (j - p < s["window"])
    scores.masked_fill_(~valid[:, None, :, None, :], -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    prob = scores.sub_(m).exp_()
    l = prob.sum(-1, keepdim=True)
    o = prob.reshape(B, Hkv, -1, k.shape[2]) @ v
    o = o.reshape(B, Hkv, -1, G, d) / torch.where(l > 0, l, 1.0)
    lse = (l.log() + m).squeeze(-1)
    # back to packed rows
    t, b = _request_of(cu, T)
    o = o.transpose(1, 2).reshape(B, -1, Hq, d)[b, t - cu[b]]
    lse = lse.transpose(1, 2).reshape(B, -1, Hq)[b, t - cu[b]]
    return o.to(q.dtype), lse.t().contiguous()


# ---------------------------------------------------------------------------
# the least that a pass has to move and compute
# ---------------------------------------------------------------------------
def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    d = case["d"]
    if case["op"] == "rope":
        rows = case["B"] * case["N"] * (case["H"] + case["Hk"])
        angles = case["N"] * case["r"] // 2
        return {"bytes": 2 * rows * d * es + 2 * case["r"] + (4 * case["N"] if case["packed"] else 0),
                "flops": 3 * rows * case["r"] + angles}
    new, cached = _lengths(case)
    T, B, Hq, Hkv, page = sum(new), case["B"], case["Hq"], case["Hkv"], case["page"]
    if case["op"] == "append_rope":
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * d * es + 8 * T + 4 * (2 * B + 1) + 2 * case["r"],
                "flops": 3 * T * (Hq + Hkv) * case["r"]}
    if case["op"] == "append8":
        pages = sum(_pages(n + c, page) - c // page for n, c in zip(new, cached))
        return {"bytes": 2 * T * Hkv * d * (es + 1) + 8 * T + 2 * 2 * 4 * pages * Hkv,
                "flops": 2 * 2 * T * Hkv * d}
    pairs = keys = scales = 0
    for n, c in zip(new, cached):
        L, W = n + c, case["window"]
        lo = max(0, c - W + 1) if W > 0 else 0   # keys that some query attends start here
        keys += L - lo
        scales += _pages(L, page) - lo // page
        for i in range(n):
            p = i + c
            a = max(0, p - W + 1) if W > 0 else 0
            z = p + 1 if case["causal"] else (min(L, p + W) if W > 0 else L)
            pairs += max(0, z - a)
    return {"bytes": 2 * keys * Hkv * d + 2 * 4 * scales * Hkv + 4 * scales + 2 * T * Hq * d * es
            + 4 * Hq * T + 4 * (2 * B + 1),
            "flops": 4 * pairs * Hq * d}


# ---------------------------------------------------------------------------
# the definition in 64 bits, token by token or request by request
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        pos = (torch.arange(case["N"], device="cuda") if s["positions"] is None
               else s["positions"][:, None])
        return tuple(_exact_rotation(x, pos, s, case["inverse"]) for x in (s["q"], s["k"]))
    new, cached = _lengths(case)
    if case["op"] == "append8":
        return _exact_append8(case, s, new, cached)
    if case["op"] == "append_rope":
        pos = torch.cat([torch.arange(c, c + n) for n, c in zip(new, cached)]).cuda()[:, None]
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        page, row = s["slots"] // s["page"], s["slots"] % s["page"]
        kc[page, :, row] = _exact_rotation(s["k"], pos, s, False)
        vc[page, :, row] = s["v"].double()
        return _exact_rotation(s["q"], pos, s, False), kc, vc
    return _exact_attend8(case, s, new, cached)


def _exact_rotation(x, pos, s, inverse):
    """Multiplication of the pairs, as complex numbers, by scaling e^(i angle)."""
    half = s["inv_freq"].numel()
    y = x.double()
    if s["interleaved"]:
        first, second = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        first, second = slice(0, half), slice(half, 2 * half)
    angle = pos.double().unsqueeze(-1) * s["inv_freq"].double()
    turn = torch.polar(torch.full_like(angle, s["scaling"]), -angle if inverse else angle)
    z = torch.complex(y[..., first], y[..., second]) * turn
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_append8(case, s, new, cached):
    """Page by page: a block's scale is the smallest power of two that holds its
    rows (those it held on the old scale, unless the page starts anew)."""
    page = case["page"]
    runs, t = [], 0   # (first token, tokens, first row, page) of each page written
    slots = s["slots"].tolist()
    for n, c in zip(new, cached):
        done = 0
        while done < n:
            row = (c + done) % page
            m = min(n - done, page - row)
            runs.append((t + done, m, row, slots[t + done] // page))
            done += m
        t += n
    if len(runs) > 3000:
        return None
    scales = torch.tensor([2.0**e for e in range(_LEAST, _MOST + 1)], dtype=torch.float64,
                          device="cuda")
    out = []
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]),
                            (s["v"], s["v_cache"], s["v_scale"])):
        q, held = cache.double(), scale.double()
        for t0, m, row, p in runs:
            rows = x[t0:t0 + m].double().transpose(0, 1)   # [Hkv, m, d]
            # the first scale that the largest value fits
            at = torch.searchsorted(_TOP * scales, rows.abs().amax((1, 2)))
            need = scales[at.clamp(max=len(scales) - 1)]
            old = held[p].clone()
            held[p] = torch.maximum(need, old) if row > 0 else need
            q[p, :, :row] = _to_e4m3(q[p, :, :row] * (old / held[p])[:, None, None])
            q[p, :, row:row + m] = _to_e4m3(rows / held[p][:, None, None])
        out.append((q, held))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _to_e4m3(x):
    """The nearest e4m3 number, ties to even: four significant bits, and
    multiples of 2^-9 below 2^-6."""
    part, power = torch.frexp(x)   # x = part 2^power, |part| in [0.5, 1)
    normal = torch.ldexp(torch.round(part * 16) / 16, power)
    small = torch.round(x * 512) / 512
    return torch.where(x.abs() >= 2.0**-6, normal, small).clamp(-_TOP, _TOP)


def _exact_attend8(case, s, new, cached):
    G, d, W = case["Hq"] // case["Hkv"], case["d"], case["window"]
    pairs = sum(n * (n + c) for n, c in zip(new, cached))
    if pairs * case["Hq"] * d > 4e11 or len(new) * case["Hq"] > 6000:
        return None
    T = sum(new)
    out = torch.zeros(T, case["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["Hq"], T), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, c) in enumerate(zip(new, cached)):
        L = n + c
        ids = s["table"][b, :_pages(L, case["page"])].long()
        kb = s["k_cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
        vb = s["v_cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
        kb, vb = (x * y[ids].double()[:, :, None, None] for x, y in ((kb, s["k_scale"]),
                                                                    (vb, s["v_scale"])))
        p = torch.arange(c, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None, :]
        bad = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        if case["causal"]:
            bad |= j > p
        if W > 0:
            bad |= p - j >= W
            if not case["causal"]:
                bad |= j - p >= W
        for hk in range(case["Hkv"]):
            K, V = kb[:, hk].reshape(-1, d)[:L], vb[:, hk].reshape(-1, d)[:L]
            for h in range(hk * G, hk * G + G):
                S = (s["q"][t0:t0 + n, h].double() @ K.t()) / math.sqrt(d)
                S[bad] = -math.inf
                z = torch.logsumexp(S, dim=1)
                lse[h, t0:t0 + n] = z
                w = torch.exp(S - torch.where(z == -math.inf, 0.0, z)[:, None])
                out[t0:t0 + n, h] = w @ V
        t0 += n
    return out, lse
