"""Rotary positions on the GPU against the definition in 64 bits, with a bound
per element: alone, as a gradient, and on the way into the paged cache."""
import math

import pytest
import torch

import exact_attention_58_gb300 as ea
from rope_fp8_ref import ref_rope, rope_tol

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def freqs(r, base=10000.0):
    return ea.attn_rope_frequencies(r, base)[0]


def check(y, x, pos, f, interleaved=False, inverse=False, scaling=1.0):
    """y against the rotation of x (CPU); untouched elements bit for bit."""
    ref = ref_rope(x, pos, f, interleaved, inverse, scaling)
    y = y.cpu()
    off = (y.double() - ref).abs() - rope_tol(x, ref, pos, f, interleaved, scaling, y.dtype)
    assert bool((off <= 0).all()), f"out of tolerance by {float(off.nan_to_num(9e9).max()):.3e}"
    r = 2 * f.numel()
    assert torch.equal(y[..., r:], x[..., r:])


def rows(*shape, dtype, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("d,r", [(64, 64), (64, 16), (128, 128), (128, 96), (256, 256), (256, 48)])
def test_dense(dtype, interleaved, inverse, d, r):
    for B, H, Hk, N in ((1, 1, 1, 1), (2, 3, 1, 37), (3, 4, 2, 130)):
        q, k = rows(B, H, N, d, dtype=dtype, seed=N), rows(B, Hk, N, d, dtype=dtype, seed=N + 1)
        f = freqs(r)
        a, b = ea.attn_rope(q.cuda(), k.cuda(), f.cuda(), interleaved=interleaved, inverse=inverse, scaling=1.25)
        for y, x in ((a, q), (b, k)):
            check(y, x, torch.arange(N), f, interleaved, inverse, 1.25)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_many_rows(dtype):
    """More rows than a thread takes, heads of both tensors, ends of tiles."""
    q, k = rows(5, 9, 67, 64, dtype=dtype), rows(5, 4, 67, 64, dtype=dtype, seed=1)
    f = freqs(64)
    for pos in (None, torch.randint(-50, 5000, (5, 67), dtype=torch.int32)):
        a, b = ea.attn_rope(q.cuda(), k.cuda(), f.cuda(), None if pos is None else pos.cuda())
        at = torch.arange(67) if pos is None else pos[:, None]
        check(a, q, at, f)
        check(b, k, at, f)
    big = rows(64, 40, 300, 64, dtype=dtype, seed=2)   # 2560 rows a position
    a, none = ea.attn_rope(big.cuda(), None, f.cuda())
    assert none is None
    check(a, big, torch.arange(300), f)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_far_positions(dtype, base):
    pos = torch.tensor([0, 1, 999, 2**17 + 3, 2**24 + 1, 2**30 - 1, 2**31 - 1, -1, -70001, -2**31], dtype=torch.int32)
    x = rows(len(pos), 2, 128, dtype=dtype)
    f = freqs(128, base)
    y, _ = ea.attn_rope(x.cuda(), None, f.cuda(), pos.cuda())
    check(y, x, pos[:, None], f)


def test_frequencies_of_any_size():
    """Above a turn per position, negative, zero."""
    f = torch.tensor([7.5, 6.2831855, 1000.25, -0.3, 0.0, 3.1415927, 1e-8, -12.0])
    x = rows(5, 1, 64, dtype=FP32)
    pos = torch.tensor([0, 1, 5, 100, 12345], dtype=torch.int32)
    y, _ = ea.attn_rope(x.cuda(), None, f.cuda(), pos.cuda())
    check(y, x, pos[:, None], f)


def test_long_context_scalings():
    for kw in (dict(method="linear"), dict(method="base"), dict(method="parts", original_len=2048)):
        f, scaling = ea.attn_rope_frequencies(64, factor=8.0, device="cuda", **kw)
        x = rows(1, 2, 200, 64, dtype=BF16)
        y, _ = ea.attn_rope(x.cuda(), None, f, scaling=scaling)
        check(y, x, torch.arange(200), f.cpu(), scaling=scaling)


def test_views_and_in_place():
    """Slices of a fused projection, heads first, a broadcast head, strided
    outputs, in place; nothing beside them is written."""
    T, H, Hk, d = 77, 5, 2, 64
    f = freqs(32).cuda()
    pos = torch.arange(1000, 1000 + T, dtype=torch.int32, device="cuda")
    fused = rows(T, H + 2 * Hk, d, dtype=BF16).cuda()
    before = fused.clone()
    q, k = fused[:, :H], fused[:, H:H + Hk]
    base = ea.attn_rope(q.contiguous(), k.contiguous(), f, pos)
    got = ea.attn_rope(q, k, f, pos)
    assert all(torch.equal(a, b) for a, b in zip(got, base)) and torch.equal(fused, before)
    out = torch.full((T, 2 * H, d), 7.0, dtype=BF16, device="cuda")
    ea.attn_rope(q, k, f, pos, q_out=out[:, ::2])
    assert torch.equal(out[:, ::2], base[0]) and bool((out[:, 1::2] == 7).all())
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(ea.attn_rope(heads_first, None, f, pos)[0], base[0])
    one = k[:, :1].expand(T, 3, d)
    assert torch.equal(ea.attn_rope(one, None, f, pos)[0], base[1][:, :1].expand(T, 3, d))
    a, b = ea.attn_rope(q, k, f, pos, q_out=q, k_out=k)
    assert a is q and b is k and torch.equal(q, base[0]) and torch.equal(k, base[1])
    assert torch.equal(fused[:, H + Hk:], before[:, H + Hk:])
    dense = rows(3, 9, 4, d, dtype=FP16).cuda().transpose(1, 2)   # [B, H, N, d] of [B, N, H, d]
    assert torch.equal(ea.attn_rope(dense, None, f)[0], ea.attn_rope(dense.contiguous(), None, f)[0])


def test_gradient():
    """Differences of the map along each input, and the formula: sum(dy . y(x))
    has the gradient that inverse=True gives."""
    f = freqs(32)
    x, dy = (rows(1, 2, 3, 64, dtype=FP32, seed=s) for s in (0, 1))
    g, _ = ea.attn_rope(dy.cuda(), None, f.cuda(), inverse=True, scaling=1.2)
    check(g, dy, torch.arange(3), f, inverse=True, scaling=1.2)
    y = lambda v: ea.attn_rope(v.cuda(), None, f.cuda(), scaling=1.2)[0].double().cpu()  # noqa: E731
    y0 = y(x)
    for at in [(0, 1, 2, 0), (0, 0, 1, 20), (0, 1, 2, 31), (0, 0, 2, 63)]:
        z = x.clone()
        z[at] += 1.0
        d = float(((y(z) - y0) * dy.double()).sum())
        # the map is linear: a step of 1 is exact but for roundings of 2^-21 of the values
        assert abs(d - float(g[at])) <= 64 * 8 * 2.0**-21


def test_around_attention():
    """A training step: rotate, attend, and the gradients back through both."""
    B, H, N, d = 1, 2, 160, 64
    f = freqs(64).cuda()
    q, k, v, do = (rows(B, H, N, d, dtype=BF16, seed=s).cuda() for s in range(4))
    rq, rk = ea.attn_rope(q, k, f)
    o, lse = ea.attn_fwd(rq, rk, v, causal=True)
    dq, dk, dv = ea.attn_bwd(rq, rk, v, o, do, lse, causal=True)
    gq, gk = ea.attn_rope(dq, dk, f, inverse=True)
    leaves = [t.double().cpu().requires_grad_() for t in (q, k, v)]
    pos = torch.arange(N)[:, None].double() * f.double().cpu()
    c, s = torch.cos(pos), torch.sin(pos)
    rot = lambda x: torch.cat((x[..., :32] * c - x[..., 32:] * s, x[..., 32:] * c + x[..., :32] * s), -1)  # noqa: E731
    S = rot(leaves[0]) @ rot(leaves[1]).transpose(2, 3) / 8.0
    S = S.masked_fill(torch.ones(N, N).triu(1).bool(), -math.inf)
    (S.softmax(-1) @ leaves[2]).backward(do.double().cpu())
    for got, leaf in zip((gq, gk, dv), leaves):
        # the attention's own bound for gradients, 5e-2 of the largest
        assert float((got.double().cpu() - leaf.grad).abs().max()) <= 5e-2 * float(leaf.grad.abs().max())


# ---------------------------------------------------------------------------
# on the way into the cache
# ---------------------------------------------------------------------------
def step(new, cached, H, Hkv, d, page, dtype, seed=0, pad=0):
    """A step's rows, empty caches, and what attn_page_table makes of the lengths."""
    T = sum(new) + pad
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    need = sum(-(-(n + c) // page) for n, c in zip(new, cached)) + 3
    width = max(-(-(n + c) // page) for n, c in zip(new, cached)) + 1
    order = torch.randperm(need, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table, at = torch.full((len(new), width), -1, dtype=torch.int32), 0
    for b, c in enumerate(cached):
        m = -(-c // page)
        table[b, :m] = order[at:at + m]
        at += m
    cu, lens, slots, _ = ea.attn_page_table(i32(cached), i32(new), table.cuda(), order[at:].cuda().contiguous(),
                                            i32([need - at]), page, T)
    q, k, v = (rows(T, n, d, dtype=dtype, seed=seed + i) for i, n in enumerate((H, Hkv, Hkv)))
    kc, vc = (torch.full((need, Hkv, page, d), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    pos = torch.cat([torch.arange(c, c + n) for n, c in zip(new, cached)] + [torch.zeros(pad, dtype=torch.int64)])
    return q, k, v, kc, vc, cu, lens, slots, pos


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r", [(64, 64), (128, 32), (256, 256)])
@pytest.mark.parametrize("new,cached", [([1] * 5, [0, 7, 100, 15, 16]), ([0, 40, 1, 0, 3], [9, 0, 70, 3, 31]),
                                        ([1, 1, 2, 1], [5, 6, 7, 8])], ids=str)
def test_append(dtype, interleaved, d, r, new, cached):
    q, k, v, kc, vc, cu, lens, slots, pos = step(new, cached, 5, 2, d, 16, dtype, pad=9)
    f = freqs(r)
    T = sum(new)
    want_k, want_v = kc.clone(), vc.clone()
    at = slots[:T].cpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    got = ea.attn_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), kc, vc, slots, f.cuda(), cu_seqlens_q=cu, seq_lens=lens,
                                    interleaved=interleaved, scaling=1.1, q_out=out, dev_status=status)
    assert got is out and int(status.item()) == 0
    check(out[:T], q[:T], pos[:T, None], f, interleaved, scaling=1.1)
    assert bool((out[T:] == 7).all())
    page, row = at // 16, at % 16
    check(kc[page, :, row], k[:T], pos[:T, None], f, interleaved, scaling=1.1)
    want_k[page, :, row] = kc[page, :, row]
    want_v[page, :, row] = v[:T].cuda()
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    # the same with positions given: all rows of q
    kc2, vc2 = torch.full_like(kc, 5.0), torch.full_like(vc, 5.0)
    out2 = ea.attn_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), kc2, vc2, slots, f.cuda(), pos.to(torch.int32).cuda(),
                                     interleaved=interleaved, scaling=1.1)
    assert torch.equal(out2[:T], out[:T]) and torch.equal(kc2, kc) and torch.equal(vc2, vc)
    check(out2[T:], q[T:], pos[T:, None], f, interleaved, scaling=1.1)


def test_append_many_requests():
    g = torch.Generator().manual_seed(4)
    new = torch.randint(0, 4, (900,), generator=g).tolist()
    cached = torch.randint(0, 500, (900,), generator=g).tolist()
    q, k, v, kc, vc, cu, lens, slots, pos = step(new, cached, 3, 1, 64, 8, BF16)
    f = freqs(64)
    out = ea.attn_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), kc, vc, slots, f.cuda(), cu_seqlens_q=cu, seq_lens=lens)
    check(out, q, pos[:, None], f)
    at = slots.cpu()
    check(kc[at // 8, :, at % 8], k, pos[:, None], f)


def test_append_bad_slots():
    """Slots of -1 are skipped, others outside the cache reported; q is rotated
    all the same; a slot of a token behind the last request is reported."""
    q, k, v, kc, vc, cu, lens, slots, pos = step([4], [10], 2, 2, 64, 16, BF16, pad=2)
    f = freqs(64)
    slots[1] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run = lambda s: ea.attn_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), kc, vc, s, f.cuda(), cu_seqlens_q=cu,  # noqa: E731
                                              seq_lens=lens, dev_status=status)
    y = run(slots)
    assert int(status.item()) == 0
    check(y[:4], q[:4], pos[:4, None], f)
    for i, bad in ((2, kc.shape[0] * 16), (2, -2), (2, 2**62), (4, 0)):
        s = slots.clone()
        s[i] = bad
        before = (kc.clone(), vc.clone())
        status.zero_()
        y = run(s)
        assert int(status.item()) == 1
        check(y[:4], q[:4], pos[:4, None], f)
        assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


def test_append_in_place_and_token_major():
    q, k, v, kc, vc, cu, lens, slots, pos = step([3, 20], [100, 0], 4, 2, 128, 16, FP16)
    f = freqs(128).cuda()
    a = ea.attn_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), kc, vc, slots, f, cu_seqlens_q=cu, seq_lens=lens)
    fused = torch.cat((q, k, v), 1).cuda()
    tm = [torch.full((kc.shape[0], 16, 2, 128), 5.0, dtype=FP16, device="cuda").transpose(1, 2) for _ in range(2)]
    b = ea.attn_cache_append_rope(fused[:, :4], fused[:, 4:6], fused[:, 6:], *tm, slots, f, cu_seqlens_q=cu, seq_lens=lens,
                                  q_out=fused[:, :4])
    assert torch.equal(a, b) and torch.equal(fused[:, :4], a) and torch.equal(fused[:, 4:].cpu(), torch.cat((k, v), 1))
    assert torch.equal(tm[0], kc) and torch.equal(tm[1], vc)


def test_captured_step():
    """A step captured with one set of lengths and replayed with another."""
    f = freqs(64).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, free, num = torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), torch.arange(16, dtype=torch.int32, device="cuda"), i32([16])
    cached, new = i32([0, 0]), i32([3, 2])
    q, k, v = (rows(5, n, 64, dtype=BF16, seed=n).cuda() for n in (4, 2, 2))
    kc, vc = (torch.zeros(16, 2, 16, 64, dtype=BF16, device="cuda") for _ in range(2))

    def once():
        cu, lens, slots, taken = ea.attn_page_table(cached, new, table, free, num, 16, 5)
        y = ea.attn_cache_append_rope(q, k, v, kc, vc, slots, f, cu_seqlens_q=cu, seq_lens=lens)
        return y, ea.attn_fwd_paged(y, kc, vc, table, lens, cu, 5, causal=True)[0]

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, o = once()
    for c, n in (([0, 0], [3, 2]), ([7, 40], [1, 4]), ([16, 1], [0, 5])):
        cached.copy_(i32(c))
        new.copy_(i32(n))
        table.fill_(-1)
        for b in range(2):
            m = -(-c[b] // 16)
            table[b, :m] = torch.arange(8 * b, 8 * b + m, dtype=torch.int32, device="cuda")
        graph.replay()
        got = y.clone(), o.clone()
        for b in range(2):   # the same once more, eagerly
            m = -(-c[b] // 16)
            table[b] = -1
            table[b, :m] = torch.arange(8 * b, 8 * b + m, dtype=torch.int32, device="cuda")
        want = once()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        pos = torch.cat([torch.arange(a, a + m) for a, m in zip(c, n)])
        check(got[0], q.cpu(), pos[:, None], f.cpu())
