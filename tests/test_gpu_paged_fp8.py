"""The paged cache held in 8 bits on the GPU: cache writes bit for bit against a
plain loop, attention against the definition in 64 bits with a bound per element."""
import math

import pytest
import torch

import exact_attention_58_gb300 as ea
from rope_fp8_ref import check_fp8, make_fp8, ref_append_fp8, to_fp8

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
NAMES = ("q", "k_cache", "v_cache", "k_scale", "v_scale", "page_table", "seq_lens", "cu")


def run(x, causal, window=0, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [kw.pop(n, getattr(x, n)) for n in NAMES]
    if kw.pop("wide", False):   # room for 64000 keys and more, unused
        args[5] = torch.nn.functional.pad(args[5], (0, 8000), value=-1)
    args = [a if a.is_cuda else a.cuda() for a in args]
    o, lse = ea.attn_fwd_paged_fp8(*args, kw.pop("max_q", x.max_q), causal=causal, window=window,
                                   dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0, f"device status {int(status.item())}"
    return o, lse


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
LENS = [
    ([1], [1]),
    ([1, 1, 1, 1], [1, 127, 128, 129]),
    ([1, 1], [1500, 40]),                      # keys split over CTAs
    ([5, 5, 5], [5, 260, 1000]),               # drafted tokens
    ([300, 1, 0, 70], [300, 513, 200, 90]),    # prompt, token, nothing new, chunk
    ([0, 40, 3], [0, 10, 0]),                  # queries before the first key, no keys at all
    ([129], [700]),
]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [(2, 2), (8, 2), (7, 1)], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_and_heads(lens, d, heads, causal):
    x = make_fp8(*lens, *heads, d, 16, seed=d + sum(lens[1]), spread=2)
    for wide in (False, True):
        check_fp8(*run(x, causal, wide=wide), x, causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 24, 48, 64, 128, 256, 384])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [40, 1, 200]], ids=str)
def test_page_sizes(d, page, q_lens):
    x = make_fp8(q_lens, [300, 129, 777], 4, 2, d, page, seed=page, spread=3)
    for wide in (False, True):
        check_fp8(*run(x, True, wide=wide), x, True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens", [[60] * 8, [1] * 8], ids=str)
def test_last_tile_of_longer_contexts(d, q_lens):
    """NaN behind the last key, whatever the ring held there before."""
    x = make_fp8(q_lens, [2700, 300, 1111, 129, 255, 2047, 513, 385], 4, 2, d, 8, seed=d)
    for _ in range(5):
        check_fp8(*run(x, True), x, True)


@pytest.mark.parametrize("window", [1, 7, 128, 300, 10**6, 2**31 - 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens", [[1, 1], [3, 2], [250, 30]], ids=str)
def test_window(window, causal, q_lens):
    x = make_fp8(q_lens, [600, 333], 4, 2, 64, 16, seed=window % 1000, spread=1)
    if causal:
        # pages that the window has left behind are given back
        for b, (n, L) in enumerate(zip(q_lens, [600, 333])):
            gone = max(0, L - n - window + 1) // 16
            lost = x.page_table[b, :gone].long()
            for c in (x.k_cache, x.v_cache):
                c.view(torch.uint8)[lost] = 0x7f
            x.k_scale[lost], x.v_scale[lost] = math.nan, -1.0
            x.page_table[b, :gone] = 2**31 - 1
    for wide in (False, True):
        check_fp8(*run(x, causal, window, wide=wide), x, causal, window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens", [[1, 1], [9, 1], [160, 2]], ids=str)
def test_fp16(d, q_lens):
    x = make_fp8(q_lens, [400, 1300], 6, 2, d, 32, dtype=FP16, seed=d, spread=1)
    for wide in (False, True):
        check_fp8(*run(x, True, wide=wide), x, True)


@pytest.mark.parametrize("heads", [(128, 1), (65, 1), (48, 1), (20, 4), (6, 2), (16, 1), (33, 1)], ids=str)
@pytest.mark.parametrize("q_lens", [[1, 1], [2, 1], [11, 40]], ids=str)
def test_groups(heads, q_lens):
    x = make_fp8(q_lens, [140, 300], *heads, 64, 16, seed=heads[0], spread=1)
    for wide in (False, True):
        check_fp8(*run(x, True, wide=wide), x, True)


@pytest.mark.parametrize("q_lens", [[1], [50], [150]], ids=str)
@pytest.mark.parametrize("what", ["keys", "scales up", "scales down", "values"])
def test_references_move(q_lens, what):
    """Row maxima, or the scales of keys or values, that keep growing or falling along
    the keys: every block asks for a new reference."""
    L, page = 1500, 16
    x = make_fp8(q_lens, [L], 4, 1, 128, page, seed=5)
    g = torch.Generator().manual_seed(6)
    ramp = torch.linspace(0.0, 1.0, L)[:, None, None]
    k, v = torch.randn(L, 1, 128, generator=g), torch.randn(L, 1, 128, generator=g)
    if what == "keys":
        k = k * (0.1 + 6 * ramp)
    elif what == "values":
        v = v * torch.exp2(40 * ramp - 20)     # 2^-20 to 2^20
    else:
        k = k * torch.exp2(24 * (ramp if what == "scales up" else 1 - ramp) - 22)
    put = make_fp8(q_lens, [L], 4, 1, 128, page, seed=5, poison=False)
    put.q = x.q
    put.k_cache, put.v_cache = (torch.zeros(put.k_cache.shape, dtype=torch.float32) for _ in range(2))
    for c in range(-(-L // page)):
        m = min(page, L - c * page)
        pg = int(put.page_table[0, c])
        put.k_cache[pg, :, :m] = k[c * page:c * page + m].transpose(0, 1)
        put.v_cache[pg, :, :m] = v[c * page:c * page + m].transpose(0, 1)
    to_fp8(put)
    for wide in (False, True):
        check_fp8(*run(put, True, wide=wide), put, True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 70])
def test_queries_of_any_size(d, q_len):
    """bf16 queries far outside fp16's range over keys as far on the other side, rows
    of zeros, rows with one large element."""
    x = make_fp8([q_len], [300], 6, 2, d, 16, seed=d)
    x.k_scale[:, 0] *= 2.0**-38          # 2^-7 and thereabouts before
    x.keys[0][:, 0] *= 2.0**-38
    x.q[:, 0] *= 2.0**38
    x.q[:, 1] *= 2.0**33
    x.q[:, 2] *= 2.0**40
    x.q[:, 3] = 0.0
    x.q[:, 4, 0] = 2.0**6
    x.q[:, 5] *= 2.0**-70
    x.q[:, 5, 1] = 1.0
    check_fp8(*run(x, True), x, True)


def test_empty_pages_of_a_new_cache():
    """A cache made of zeros: scales of 0 stand for 2^-48 and are not reported."""
    x = make_fp8([1, 40], [100, 90], 4, 2, 64, 16, poison=False)
    x.k_cache, x.v_cache = (torch.zeros(x.k_cache.shape).to(torch.float8_e4m3fn) for _ in range(2))
    x.k_scale.zero_()
    x.v_scale.zero_()
    for b in range(2):
        x.keys[b].zero_()
        x.values[b].zero_()
    check_fp8(*run(x, True), x, True)


@pytest.mark.parametrize("q_len", [1, 100])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_bad_scales_are_reported(q_len, which):
    """No power of two: reported, and its exponent counts.  Pages outside the
    cache are reported too, and zeros read."""
    for bad in (3.0, -1.0, math.nan, math.inf):
        x = make_fp8([q_len], [300], 4, 2, 64, 16)
        getattr(x, which)[int(x.page_table[0, 5]), 1] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ea.attn_fwd_paged_fp8(*(getattr(x, n).cuda() for n in NAMES), x.max_q, causal=True, dev_status=status)
        assert int(status.item()) == 1
    x = make_fp8([q_len], [300], 4, 2, 64, 16)
    for page in (-1, x.k_cache.shape[0], 2**31 - 1):
        y = make_fp8([q_len], [300], 4, 2, 64, 16)
        y.page_table[0, 7] = page
        y.keys[0][112:128], y.values[0][112:128] = 0.0, 0.0
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = ea.attn_fwd_paged_fp8(*(getattr(y, n).cuda() for n in NAMES), y.max_q, causal=True, dev_status=status)
        assert int(status.item()) == 1
        check_fp8(o, lse, y, True)


@pytest.mark.parametrize("q_len", [1, 40])
def test_nan_that_is_attended(q_len):
    """A NaN key or value reaches the rows that attend it, and no other head's."""
    for which in ("k_cache", "v_cache"):
        x = make_fp8([q_len], [300], 4, 2, 64, 16)
        pg = int(x.page_table[0, 3])
        getattr(x, which).view(torch.uint8)[pg, 0, 5, 7] = 0x7f
        o, lse = run(x, True)
        hit = o[:, :2, 7] if which == "v_cache" else o[:, :2]
        assert bool(hit.isnan().all()) and not bool(o[:, 2:].isnan().any())


@pytest.mark.parametrize("q_lens", [[1, 1, 0], [40, 1, 130]], ids=str)
def test_rows_behind_the_last_sequence_are_left(q_lens):
    x = make_fp8(q_lens, [200, 5, 400], 4, 2, 64, 16, seed=1, extra_rows=37)
    x.q[sum(q_lens):] = math.nan
    out = torch.full(x.q.shape, 7.0, dtype=BF16, device="cuda")
    lse = torch.full((4, x.q.shape[0]), 7.0, device="cuda")
    run(x, True, out=out, lse=lse)
    check_fp8(out, lse, x, True)
    T = sum(q_lens)
    assert bool((out[T:] == 7).all()) and bool((lse[:, T:] == 7).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 4, 150])
def test_strided_views(q_len, d):
    """Queries as a slice of a fused projection; token-major pages; K and V side
    by side in one array."""
    H, Hkv, page = 4, 2, 16
    x = make_fp8([q_len, 1], [500, 77], H, Hkv, d, page, seed=q_len)
    fused = torch.full((q_len + 1, H + 2 * Hkv, d), math.nan, dtype=BF16)
    fused[:, :H] = x.q
    base = run(x, True)
    check_fp8(*base, x, True)
    u8 = lambda t: t.view(torch.uint8)  # noqa: E731
    kv = torch.stack([u8(x.k_cache), u8(x.v_cache)], 1).cuda().view(torch.float8_e4m3fn)
    tm = [u8(t).transpose(1, 2).contiguous().cuda().transpose(1, 2).view(torch.float8_e4m3fn)
          for t in (x.k_cache, x.v_cache)]
    for kc, vc in ((kv[:, 0], kv[:, 1]), tm):
        assert not kc.is_contiguous()
        o, lse = run(x, True, q=fused.cuda()[:, :H], k_cache=kc, v_cache=vc)
        assert torch.equal(o, base[0]) and torch.equal(lse, base[1])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_tiles(d):
    """Several rounds of query tiles per CTA, uniform and ragged, with and
    without a window."""
    for q_lens, k_lens in (([130] * 40, [200] * 40), ([0, 300, 1, 77] * 10, [50, 350, 400, 90] * 10)):
        x = make_fp8(q_lens, k_lens, 8, 8, d, 16, seed=d, spread=1)
        check_fp8(*run(x, True), x, True)
        check_fp8(*run(x, False, 60), x, False, 60)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (65, 1)], ids=str)
def test_single_tokens_beside_a_chunk(d, heads):
    """Short requests and long ones in one call, which go to a kernel each: every row
    is written once."""
    group = heads[0] // heads[1]
    q_lens = [1] * 14 + [150] + [16 // group, 0, 16 // group + 1, 64 // group + 1] + [2] * 6
    k_lens = [37 * i + q + 5 for i, q in enumerate(q_lens)]
    k_lens[3], k_lens[20] = 0, 1
    x = make_fp8(q_lens, k_lens, *heads, d, 16, seed=d, extra_rows=3)
    for wide in (False, True):
        out = torch.full(x.q.shape, 7.0, dtype=BF16, device="cuda")
        lse = torch.full((heads[0], x.q.shape[0]), 7.0, device="cuda")
        run(x, True, 90, wide=wide, out=out, lse=lse)
        check_fp8(out, lse, x, True, 90)
        assert bool((out[-3:] == 7).all()) and bool((lse[:, -3:] == 7).all())


def test_many_requests():
    g = torch.Generator().manual_seed(3)
    k_lens = torch.randint(0, 300, (700,), generator=g).tolist()
    q_lens = [min(1, n) for n in k_lens]
    x = make_fp8(q_lens, k_lens, 2, 1, 64, 16, seed=9)
    check_fp8(*run(x, True), x, True)


@pytest.mark.parametrize("longest,max_q", [(200, 200), (2, 200), (0, 2)])
@pytest.mark.parametrize("B", [8, 40])
def test_mostly_empty_batches(longest, max_q, B):
    q_lens = ([0, 0, longest] + [0] * 5) * (B // 8)
    rows = sum(q_lens) + 9
    x = make_fp8(q_lens, [500 + q for q in q_lens], 4, 2, 64, 16, seed=1, extra_rows=9)
    for wide in (False, True):
        out = torch.full((rows, 4, 64), 7.0, dtype=BF16, device="cuda")
        lse = torch.full((4, rows), 7.0, device="cuda")
        run(x, True, max_q=max_q, wide=wide, out=out, lse=lse)
        check_fp8(out, lse, x, True)
        assert bool((out[-9:] == 7).all()) and bool((lse[:, -9:] == 7).all())


@pytest.mark.parametrize("q_len", [1, 3, 90])
def test_guard_bands(q_len):
    """Nothing is written outside O and LSE, nor to the cache; max_seqlen_q is a bound."""
    x = make_fp8([q_len, 1, 7], [300, 90, 40], 4, 2, 64, 16, seed=3)
    n, band = x.q.numel(), 4096
    buf = torch.full((n + 2 * band,), 3.0, dtype=BF16, device="cuda")
    lbuf = torch.full((4 * x.q.shape[0] + 2 * band,), 3.0, device="cuda")
    out, lse = buf[band:band + n].view(x.q.shape), lbuf[band:-band].view(4, -1)
    for kw in (dict(), dict(wide=True), dict(max_q=1000)):
        run(x, True, out=out, lse=lse, **kw)
        check_fp8(out, lse, x, True)
        for b in (buf, lbuf):
            assert bool((b[:band] == 3).all()) and bool((b[-band:] == 3).all())


def test_two_streams_and_a_dirty_workspace():
    """Calls with a workspace each on two streams at the same time; one whose
    workspace holds NaN on entry, and an own scale."""
    a = make_fp8([1] * 5, [3000, 100, 900, 2000, 50], 8, 2, 128, 16, seed=50)
    b = make_fp8([300, 40], [1300, 700], 8, 2, 128, 16, seed=51)
    ref = [run(x, True, wide=True) for x in (a, b)]
    dev = []
    for x in (a, b):
        t = [getattr(x, n).cuda() for n in NAMES]
        t[5] = torch.nn.functional.pad(t[5], (0, 8000), value=-1)
        dev.append(t)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(10):
        for i, x in enumerate((a, b)):
            got[i].append(ea.attn_fwd_paged_fp8(*dev[i], x.max_q, causal=True, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, ref[i][0]) and torch.equal(lse, ref[i][1])
    n = ea.attn_fwd_paged_workspace_size(5, 8, 2, 5, 1, a.page_table.shape[1] + 8000, 16, 128)
    assert n > 0
    ws = torch.full((n // 4 + 1,), math.nan, device="cuda")
    check_fp8(*run(a, True, scale=0.3, workspace=ws, wide=True), a, True, scale=0.3)


def test_cache_past_32_bit_offsets():
    """Pages more than 2^32 elements into the pool."""
    page, Hkv, d = 64, 8, 128
    num_pages = 2**32 // (page * Hkv * d) + 50
    x = make_fp8([1, 70], [500, 200], 16, Hkv, d, page, seed=6)
    kc, vc = (torch.zeros(num_pages, Hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(num_pages, Hkv, device="cuda") for _ in range(2))
    table, mine = x.page_table.clone(), x.page_table >= 0
    used = x.page_table[mine].long()
    there = used + num_pages - x.k_cache.shape[0]
    table[mine] = there.to(torch.int32)
    for big, small in ((kc, x.k_cache.view(torch.uint8)), (vc, x.v_cache.view(torch.uint8)), (ks, x.k_scale), (vs, x.v_scale)):
        big[there.cuda()] = small[used].cuda()
    check_fp8(*run(x, True, k_cache=kc.view(torch.float8_e4m3fn), v_cache=vc.view(torch.float8_e4m3fn), k_scale=ks,
                   v_scale=vs, page_table=table), x, True)
    # and the append's
    k = torch.randn(3, Hkv, d, generator=torch.Generator().manual_seed(1)).to(BF16)
    slots = torch.arange(3, dtype=torch.int64) + (num_pages - 1) * page + 8
    ref, exps = kc[-1:].view(torch.float8_e4m3fn).double().cpu(), torch.frexp(ks[-1:].cpu()).exponent.long() - 1
    ea.attn_cache_append_fp8(k.cuda(), k.cuda(), kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs, slots.cuda())
    ref_append_fp8(k, ref, exps, [8, 9, 10], page)
    assert torch.equal(kc[-1:].view(torch.float8_e4m3fn).double().cpu().nan_to_num(1e9), ref.nan_to_num(1e9))
    assert torch.equal(torch.frexp(ks[-1:].cpu()).exponent.long() - 1, exps)


# ---------------------------------------------------------------------------
# cache writes
# ---------------------------------------------------------------------------
def append_and_check(runs, Hkv, d, page, pages, dtype=BF16, seed=0, factor=None, poison=True):
    """Appends each (slots, factor) in turn and compares the caches bit for bit."""
    g = torch.Generator().manual_seed(seed)
    kc, vc = (torch.full((pages, Hkv, page, d), 0x7f if poison else 0, dtype=torch.uint8) for _ in range(2))
    ref = [c.view(torch.float8_e4m3fn).double() for c in (kc, vc)]
    exps = [torch.zeros(pages, Hkv, dtype=torch.int64) for _ in range(2)]
    caches = [c.cuda().view(torch.float8_e4m3fn) for c in (kc, vc)]
    scales = [torch.ones(pages, Hkv, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for slots, factor in runs:
        k, v = ((torch.randn(len(slots), Hkv, d, generator=g) * factor).to(dtype) for _ in range(2))
        v = v * 8
        ea.attn_cache_append_fp8(k.cuda(), v.cuda(), *caches, *scales, torch.tensor(slots, device="cuda"), dev_status=status)
        for x, c, e in zip((k, v), ref, exps):
            ref_append_fp8(x, c, e, slots, page)
        for c, s, rc, re in zip(caches, scales, ref, exps):
            assert torch.equal(torch.exp2(re.double()).float(), s.cpu())
            assert torch.equal(c.double().cpu().nan_to_num(1e9), rc.nan_to_num(1e9))
        assert int(status.item()) == 0
    return caches, scales


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 24, 128, 384])
def test_append(dtype, d, page):
    """Prompts over several pages, then tokens and chunks that continue pages, with
    larger and smaller values, then a page written anew."""
    first = list(range(3 * page, 5 * page + 5)) + list(range(page, page + 3))
    more = [5 * page + 5, page + 3, page + 4, -1, 7 * page]
    append_and_check([(first, 1.0), (more, 30.0), ([5 * page + 6, page + 5], 0.01), ([x + 1 for x in more[:1]], 1000.0),
                      (list(range(3 * page, 3 * page + 4)), 0.1), ([-1, -1, 4 * page + 1], 3e4 if dtype is BF16 else 100.0)],
                     3, d, page, 9, dtype, seed=page + d)


def test_append_single_tokens():
    """Token by token through a page and into the next, as decoding does."""
    append_and_check([([40 + i, 7 - i % 8 + 144], 2.0 ** (i % 5)) for i in range(30)], 2, 64, 8, 20, seed=1)


def test_append_many():
    """More runs than CTAs, of every length, pages in any order."""
    g = torch.Generator().manual_seed(2)
    pages = torch.randperm(700, generator=g).tolist()
    slots = []
    for i, p in enumerate(pages[:600]):
        r = int(torch.randint(0, 16, (1,), generator=g))
        n = int(torch.randint(1, 17 - r, (1,), generator=g))
        slots += [p * 16 + r + j for j in range(n)] + [-1] * (i % 3 == 0)
    append_and_check([(slots, 1.0)], 4, 64, 16, 700)


def test_append_special_values():
    """Zeros, infinities, NaN, the smallest and largest numbers; a block of zeros
    takes the smallest scale; a page of an old cache whose scale is 0."""
    page = 8
    for dtype in (BF16, FP16):
        info = torch.finfo(dtype)
        x = torch.zeros(6, 1, 64, dtype=dtype)
        x[1, 0, :6] = torch.tensor([info.max, -info.max, info.tiny, 1.0, math.inf, -math.inf])
        x[2, 0, 3] = math.nan
        x[3, 0, :2] = torch.tensor([448.0, 1.0])
        x[4, 0, 0], x[5] = 449.0, info.tiny
        for rows, slots in (([0], [8]), ([1], [16]), ([2], [24]), ([3], [32]), ([4], [40]), ([5], [48]), ([2, 3], [58, 59]),
                            ([0, 5], [65, 66])):
            kc = torch.zeros(9, 1, page, 64).to(torch.float8_e4m3fn)
            ref, exps = kc.double(), torch.full((9, 1), -48)
            c, s = kc.cuda(), torch.zeros(9, 1, device="cuda")
            c2, s2 = kc.cuda(), torch.zeros(9, 1, device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            k = x[rows].contiguous()
            ea.attn_cache_append_fp8(k.cuda(), k.cuda(), c, c2, s, s2, torch.tensor(slots, device="cuda"), dev_status=status)
            ref_append_fp8(k, ref, exps, slots, page)
            p = slots[0] // page
            assert float(s[p, 0]) == 2.0 ** int(exps[p, 0]) and float(s.sum()) == float(s[p, 0])
            assert torch.equal(c.double().cpu().nan_to_num(1e9), ref.nan_to_num(1e9)) and int(status.item()) == 0
            assert torch.equal(c2.view(torch.uint8), c.view(torch.uint8)) and torch.equal(s2, s)


def test_append_reports():
    """Slots outside the cache, and a continued block whose scale is no power of two."""
    k = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(0)).to(BF16).cuda()
    new = lambda: [torch.zeros(4, 2, 8, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)] + [torch.ones(4, 2, device="cuda") for _ in range(2)]  # noqa: E731
    for slots, scale, want in (([1, -1, 9], 1.0, 0), ([1, 32, 9], 1.0, 1), ([1, -2, 9], 1.0, 1), ([2**40, 2**62, -2**63], 1.0, 1),
                               ([1, 2, 9], 0.0, 0), ([1, 2, 9], 3.0, 1), ([1, 2, 9], math.nan, 1), ([8, 9, 10], math.nan, 0)):
        c = new()
        c[2].fill_(scale)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ea.attn_cache_append_fp8(k, k, *c, torch.tensor(slots, device="cuda"), dev_status=status)
        assert int(status.item()) == want, (slots, scale)
        good = [(t, s) for t, s in enumerate(slots) if 0 <= s < 32]
        touched = {(s // 8, s % 8) for _, s in good}
        for p in range(4):
            for r in range(8):
                if (p, r) not in touched:
                    assert not bool(c[0].view(torch.uint8)[p, :, r].any())


def test_append_strided():
    """k and v as slices of a fused projection, token-major pages; neighbours stay."""
    x = torch.randn(20, 8, 64, generator=torch.Generator().manual_seed(0)).to(FP16).cuda()
    slots = torch.arange(5, 25, device="cuda")
    a = [torch.zeros(4, 2, 8, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    b = [torch.full((4, 8, 3, 64), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sa, sb = ([torch.ones(4, 2, device="cuda") for _ in range(2)] for _ in range(2))
    for t in b:
        t[:, :, :2] = 0
    ea.attn_cache_append_fp8(x[:, 4:6].contiguous(), x[:, 6:].contiguous(), *a, *sa, slots)
    ea.attn_cache_append_fp8(x[:, 4:6], x[:, 6:], *(t.transpose(1, 2)[:, :2].view(torch.float8_e4m3fn) for t in b), *sb, slots)
    for c, t, s, u in zip(a, b, sa, sb):
        assert torch.equal(c.view(torch.uint8), t.transpose(1, 2)[:, :2]) and torch.equal(s, u)
        assert bool((t[:, :, 2] == 9).all())


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("heads", [(4, 2), (7, 1)], ids=str)
def test_decoding_loop(heads):
    """A prompt in two chunks, then tokens: page table, rotation, append to the
    8-bit cache and attention, against the same in 64 bits from what the cache holds."""
    H, Hkv = heads
    d, page, dev = 64, 16, "cuda"
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    g = torch.Generator().manual_seed(7)
    f, _ = ea.attn_rope_frequencies(d, device=dev)
    kc, vc = (torch.zeros(40, Hkv, page, d, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(40, Hkv, device=dev) for _ in range(2))
    table, status = torch.full((2, 20), -1, dtype=torch.int32, device=dev), i32(0)
    free, num_free, cached = torch.randperm(40, generator=g).to(torch.int32).cuda(), i32(40), i32(0, 0)
    pages = [torch.zeros(40, Hkv, page, d, dtype=torch.float64) for _ in range(2)]
    exps = [torch.zeros(40, Hkv, dtype=torch.int64) for _ in range(2)]
    for new in ([130, 33], [70, 1], [1, 1], [1, 5], [1, 1]):
        T = sum(new)
        cu, lens, slots, taken = ea.attn_page_table(cached, i32(*new), table, free, num_free, page, T, dev_status=status)
        q, k, v = (torch.randn(T, n, d, generator=g).to(BF16).cuda() for n in (H, Hkv, Hkv))
        pos = torch.cat([torch.arange(c, c + n) for c, n in zip(cached.tolist(), new)]).to(torch.int32).cuda()
        q, k = ea.attn_rope(q, k, f, pos)
        ea.attn_cache_append_fp8(k, v, kc, vc, ks, vs, slots, dev_status=status)
        for x, c, e in ((k, pages[0], exps[0]), (v, pages[1], exps[1])):
            ref_append_fp8(x.cpu(), c, e, slots.tolist(), page)
        for c, s, rc, e in ((kc, ks, pages[0], exps[0]), (vc, vs, pages[1], exps[1])):
            held = torch.unique(table[table >= 0].long()).cpu()
            assert torch.equal(s.cpu()[held], torch.exp2(e.double()).float()[held])
            assert torch.equal(c.double().cpu()[held], rc[held])
        o, lse = ea.attn_fwd_paged_fp8(q, kc, vc, ks, vs, table, lens, cu, max(new), causal=True, dev_status=status)
        x = make_fp8(new, lens.tolist(), H, Hkv, d, page, poison=False)
        x.q, x.page_table, x.k_scale, x.v_scale = q.cpu(), table.cpu(), ks.cpu(), vs.cpu()
        for b, L in enumerate(lens.tolist()):
            ids = table[b, :-(-L // page)].long().cpu()
            for lists, c, e in ((x.keys, pages[0], exps[0]), (x.values, pages[1], exps[1])):
                lists[b] = (c[ids] * torch.exp2(e[ids].double())[:, :, None, None]).transpose(1, 2).reshape(-1, Hkv, d)[:L]
        check_fp8(o, lse, x, True)
        cached, num_free = lens, num_free - taken
    assert int(status.item()) == 0


def test_captured_step():
    """Append and attention captured with one set of lengths, replayed with others."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    dev, d, Hkv = "cuda", 128, 2
    table = torch.arange(64, dtype=torch.int32, device=dev).view(2, 32)
    cached, new = i32([0, 0]), i32([1, 1])
    free, num = torch.zeros(1, dtype=torch.int32, device=dev), i32([0])
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(2, n, d, generator=g).to(BF16).cuda() for n in (8, Hkv, Hkv))
    start = torch.randint(0, 0x70, (2, 64, Hkv, 16, d), generator=g, dtype=torch.uint8).cuda()

    def fresh():
        return [t.clone().view(torch.float8_e4m3fn) for t in start] + [torch.full((64, Hkv), 2.0**-8, device=dev) for _ in range(2)]

    c = fresh()

    def once(kc, vc, ks, vs):
        cu, lens, slots, _ = ea.attn_page_table(cached, new, table, free, num, 16, 2)
        ea.attn_cache_append_fp8(k, v, kc, vc, ks, vs, slots)
        return ea.attn_fwd_paged_fp8(q, kc, vc, ks, vs, table, lens, cu, 1, causal=True)

    cached.copy_(i32([3, 3]))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        once(*c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = once(*c)
    for lens in ([5, 300], [511, 17], [100, 101]):
        lens = [n if n % 16 else n + 1 for n in lens]
        cached.copy_(i32(lens))
        for t, s in zip(c, fresh()):
            t.copy_(s)
        graph.replay()
        got = o.clone(), lse.clone(), [t.clone() for t in c]
        e = fresh()
        want = once(*e)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for a, b in zip(got[2], e):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_same_result_every_time():
    x = make_fp8([1] * 7 + [4], [4000, 33, 800, 1, 129, 2500, 64, 900], 8, 2, 128, 16, seed=8)
    for wide in (False, True):
        a = run(x, True, wide=wide)
        for _ in range(3):
            b = run(x, True, wide=wide)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
