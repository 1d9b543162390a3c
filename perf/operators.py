"""The serving operators over a paged key/value cache, as workloads to time.

Three operators: ``attn_page_table`` (page table and slot map of one serving
step), ``attn_cache_append`` (new key and value rows into their slots) and
``attn_fwd_paged`` (attention of new tokens over the cache).  ``run`` computes
them in plain torch operations, or through the package where ``own`` is true.
A case holds plain values; its request lengths come from its own
``lens_seed``, the tensors' values and the page order from the seed given to
``prepare``.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attend(name, B, q, ctx, Hq, Hkv, d, page, dtype="bf16", causal=True, window=0, lens_seed=1):
    return {"name": name, "op": "attend", "B": B, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype,
            "causal": causal, "window": window, "lens_seed": lens_seed}


def _append(name, B, q, ctx, Hkv, d, page, dtype="bf16", lens_seed=1):
    return {"name": name, "op": "append", "B": B, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hkv": Hkv, "d": d, "page": page, "dtype": dtype,
            "lens_seed": lens_seed}


def _table(name, B, q, ctx, page, pad, lens_seed=1):
    return {"name": name, "op": "table", "B": B, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "page": page, "pad": pad, "lens_seed": lens_seed}


def listed():
    return [
        # One interactive request of a 12-head, d = 64 model writing its next
        # token: latency.
        _attend("token_b1_h12_d64", 1, (1, 1), (997, 997), 12, 12, 64, 16),
        # A serving batch, one token per request, ragged contexts, four query
        # heads to a key head: bound by reading the cache.
        _attend("token_b48_h32kv8_d128", 48, (1, 1), (130, 4200), 32, 8, 128, 16, lens_seed=2),
        # Two very long contexts with few key heads: the keys have to be split
        # over the whole GPU.
        _attend("token_long_b2_h16kv2_d128", 2, (1, 1), (70001, 131072), 16, 2, 128, 64,
                lens_seed=3),
        # Five drafted tokens and the last accepted one checked in one pass;
        # seven query heads to a key head, fp16.
        _attend("verify6_b17_h28kv4_d128", 17, (6, 6), (300, 6000), 28, 4, 128, 32, dtype="fp16",
                lens_seed=4),
        # A chunk of a long prompt over what is already cached.
        _attend("chunk512_b1_h16_d128", 1, (512, 512), (16100, 16100), 16, 16, 128, 64),
        # A mixed step: prompt chunks beside single tokens, sliding window,
        # odd page size.
        _attend("mixed_b12_h16kv4_d64_window", 12, (1, 700), (0, 3500), 16, 4, 64, 48,
                window=1024, lens_seed=6),
        # Short chunks at head dim 256, eight tokens a page.
        _attend("chunk_b8_h8kv4_d256", 8, (33, 65), (500, 2700), 8, 4, 256, 8, lens_seed=7),
        # Whole prompts at the 4 x 16 x 4096 x 128 causal shape.
        _attend("prompt_b4_h16_n4096_d128", 4, (4096, 4096), (0, 0), 16, 16, 128, 128),
        # The new rows of one decoding step, and of one step of prompt chunks.
        _append("append_token_b64", 64, (1, 1), (100, 5000), 8, 128, 16),
        _append("append_prompt_b16", 16, (900, 1100), (0, 1000), 8, 128, 64, lens_seed=2),
        # The tables of a decoding step, and of a large mixed step whose token
        # buffer is padded.
        _table("table_token_b48", 48, (1, 1), (130, 4200), 16, 0),
        _table("table_mixed_b512", 512, (1, 250), (0, 9000), 16, 1000, lens_seed=2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "table"])
    seed = rng.randrange(1 << 30)
    page = rng.choice([8, 16, 16, 32, 48, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "table":
        q_hi = rng.choice([1, 1, _log_int(rng, 2, 250)])
        ctx_hi = _log_int(rng, 10, 9000)
        case = _table(None, _log_int(rng, 1, 512), (1, q_hi), (0, ctx_hi), page,
                      rng.choice([0, rng.randrange(1000)]), seed)
    elif op == "append":
        q_hi = rng.choice([1, _log_int(rng, 2, 1100)])
        B = _log_int(rng, 1, 64 if q_hi < 250 else 16)
        case = _append(None, B, (1, q_hi), (0, _log_int(rng, 10, 5000)),
                       rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), page, dtype, seed)
    else:
        d = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8, 12, 16])
        G = rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
        kind = rng.choice(["token", "verify", "chunk", "prompt"])
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
            q_hi = _log_int(rng, 100, 4096)
            q, ctx_hi, B = (max(1, q_hi // 2), q_hi), 1, _log_int(rng, 1, 8)
        while G > 1 and Hkv * G > 32:
            G -= 1
        # no more products than the 4 x 16 x 4096 x 128 shape, and no more
        # cached elements than a 48 x 4200 x 8 x 128 cache, padded
        while B > 1 and (B * Hkv * G * q[1] * (q[1] + ctx_hi) * d > 4 * 16 * 4096 * 4096 * 128
                         or B * Hkv * (q[1] + ctx_hi) * d > 48 * 4200 * 8 * 128):
            B -= 1
        while Hkv * (q[1] + ctx_hi) * d > 48 * 4200 * 8 * 128 and Hkv > 1:
            Hkv //= 2
        case = _attend(None, B, q, (ctx_hi // 3, ctx_hi), Hkv * G, Hkv, d, page, dtype, causal,
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
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new, cached = _lengths(case)
    lens = [n + c for n, c in zip(new, cached)]
    page, B, T = case["page"], case["B"], sum(new)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    # Pages in the order in which a busy pool hands them out: any.
    filled = [_pages(x, page) for x in lens]
    num_pages = sum(filled) + max(2, sum(filled) // 8)
    order = torch.randperm(num_pages, device="cuda", generator=gen).to(torch.int32)
    # Before attn_page_table a request holds the pages of its cached tokens
    # only; the row has room for the longest request and a few pages more.
    table_op = case["op"] == "table"
    holds = [_pages(c, page) for c in cached] if table_op else filled
    width = max(filled) + (3 if table_op else 0)
    starts = torch.tensor([0] + holds[:-1], device="cuda").cumsum(0)
    col = torch.arange(width, device="cuda")
    page_table = torch.where(col < torch.tensor(holds, device="cuda")[:, None],
                             order[(starts[:, None] + col).clamp(max=num_pages - 1)],
                             -1).to(torch.int32).contiguous()
    s = {"op": case["op"], "page": page, "page_table": page_table}
    if table_op:
        free = num_pages - sum(holds)
        free_pages = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
        free_pages[:free] = order[sum(holds):]
        s.update(cached_lens=i32(cached), new_lens=i32(new), free_pages=free_pages,
                 num_free=i32([free]), max_tokens=T + case["pad"])
        return s

    dtype, Hkv, d = _DTYPES[case["dtype"]], case["Hkv"], case["d"]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).to(dtype)

    # [pages, key heads, tokens of a page, d]; slots that hold no token keep
    # what was in them.
    s["k_cache"] = randn(num_pages, Hkv, page, d)
    s["v_cache"] = randn(num_pages, Hkv, page, d)
    cu = i32([0] + new).cumsum(0).to(torch.int32)
    if case["op"] == "append":
        s["k"], s["v"] = randn(T, Hkv, d), randn(T, Hkv, d)
        b = torch.repeat_interleave(torch.arange(B, device="cuda"),
                                    torch.tensor(new, device="cuda"))
        pos = torch.arange(T, device="cuda") - cu.long()[b] + i32(cached).long()[b]
        s["slots"] = page_table[b, pos // page].long() * page + pos % page
        return s
    s.update(q=randn(T, case["Hq"], d), cu=cu, seq_lens=i32(lens), max_q=max(new), max_k=max(lens),
             causal=case["causal"], window=case["window"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return {"attend": _run_attend, "append": _run_append, "table": _run_table}[state["op"]](state)


def _run_attend(s):
    if own:
        import exact_attention_58_gb300 as ea
        return ea.attn_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"],
                                 s["seq_lens"], s["cu"], s["max_q"], causal=s["causal"],
                                 window=s["window"])
    q, cu, seq_lens = s["q"], s["cu"].long(), s["seq_lens"].long()
    T, Hq, d = q.shape
    _, Hkv, page, _ = s["k_cache"].shape
    B, G, dev = cu.numel() - 1, Hq // Hkv, q.device
    ids = s["page_table"][:, :_pages(s["max_k"], page)].clamp(min=0).long()
    # [B, Hkv, keys, d]
    k = s["k_cache"][ids].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    v = s["v_cache"][ids].transpose(1, 2).reshape(B, Hkv, -1, d).float()
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
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    o = o.transpose(1, 2).reshape(B, -1, Hq, d)[b, t - cu[b]]
    lse = lse.transpose(1, 2).reshape(B, -1, Hq)[b, t - cu[b]]
    return o.to(q.dtype), lse.t().contiguous()


def _run_append(s):
    if own:
        import exact_attention_58_gb300 as ea
        ea.attn_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
        return s["k_cache"], s["v_cache"]
    page, row = s["slots"] // s["page"], s["slots"] % s["page"]
    s["k_cache"][page, :, row] = s["k"]
    s["v_cache"][page, :, row] = s["v"]
    return s["k_cache"], s["v_cache"]


def _run_table(s):
    table = s["page_table"]
    if own:
        import exact_attention_58_gb300 as ea
        cu, seq_lens, slots, taken = ea.attn_page_table(
            s["cached_lens"], s["new_lens"], table, s["free_pages"], s["num_free"], s["page"],
            s["max_tokens"])
        return cu, seq_lens, slots, taken, table
    page, cached, new = s["page"], s["cached_lens"].long(), s["new_lens"].long()
    dev = table.device
    ends = new.cumsum(0)
    cu = torch.cat([ends.new_zeros(1), ends])
    seq_lens = cached + new
    held = (cached + page - 1) // page
    need = (seq_lens + page - 1) // page - held
    first = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=dev)
    nth = first[:, None] + col - held[:, None]
    taken_from = (s["num_free"] - 1 - nth).clamp(0, s["free_pages"].numel() - 1)
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    table.copy_(torch.where(fresh, s["free_pages"][taken_from], table))
    t = torch.arange(s["max_tokens"], device=dev)
    b = torch.searchsorted(ends, t, right=True).clamp(max=table.shape[0] - 1)
    pos = cached[b] + t - cu[b]
    at = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(t < ends[-1], at * page + pos % page, -1)
    return (cu.to(torch.int32), seq_lens.to(torch.int32), slots,
            need.sum().reshape(1).to(torch.int32), table)


# ---------------------------------------------------------------------------
# the least that a pass has to move and compute
# ---------------------------------------------------------------------------
def work(case):
    new, cached = _lengths(case)
    page, T, B = case["page"], sum(new), case["B"]
    if case["op"] == "table":
        fresh = sum(_pages(n + c, page) - _pages(c, page) for n, c in zip(new, cached))
        kept = sum(1 for c in cached if c % page)   # the page that a request's new tokens continue
        return {"bytes": 4 * (2 * B + 1) + 4 * (fresh + kept) + 4 * (2 * B + 1) + 4 * fresh + 4
                + 8 * (T + case["pad"]),
                "flops": 4 * B + 3 * T}
    row = case["Hkv"] * case["d"] * 2
    if case["op"] == "append":
        return {"bytes": 4 * T * row + 8 * T, "flops": 0}
    keys = pairs = 0
    W, causal = case["window"], case["causal"]
    for n, c in zip(new, cached):
        L = n + c
        lo, hi = 0, L
        if W > 0:   # the first query's window reaches furthest back
            lo = max(0, c - W + 1)
        keys += hi - lo
        for i in range(n):
            p = c + i
            last = min(L - 1, p) if causal else (min(L - 1, p + W - 1) if W > 0 else L - 1)
            first = max(0, p - W + 1) if W > 0 else 0
            pairs += last - first + 1
    tables = sum(_pages(n + c, page) for n, c in zip(new, cached))
    io = 2 * T * case["Hq"] * case["d"] * 2 + 4 * T * case["Hq"]
    return {"bytes": 2 * keys * row + io + 4 * tables + 4 * (2 * B + 1),
            "flops": 4 * case["Hq"] * case["d"] * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] != "attend":
        return None   # whole numbers, copies
    s = prepare(case, seed)
    new, cached = _lengths(case)
    page = case["page"]
    T, Hq, d = s["q"].shape
    Hkv = case["Hkv"]
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, c) in enumerate(zip(new, cached)):
        L = n + c
        ids = s["page_table"][b, :_pages(L, page)].tolist()
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            K = s["k_cache"][ids, kv].reshape(-1, d)[:L].double()
            V = s["v_cache"][ids, kv].reshape(-1, d)[:L].double()
            S = (s["q"][t0:t0 + n, h].double() @ K.t()) / math.sqrt(d)
            p = torch.arange(c, L, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")[None, :]
            bad = torch.zeros_like(S, dtype=torch.bool)
            if case["causal"]:
                bad |= j > p
            if case["window"] > 0:
                bad |= p - j >= case["window"]
                if not case["causal"]:
                    bad |= j - p >= case["window"]
            S[bad] = -math.inf
            z = torch.logsumexp(S, dim=1)
            lse[h, t0:t0 + n] = z
            w = torch.exp(S - torch.where(z == -math.inf, 0.0, z)[:, None])
            out[t0:t0 + n, h] = w @ V
        t0 += n
    return out, lse
