"""Serving from a paged key/value cache on the GPU: attention against the
definition in 64 bits with an error bound per element, cache writes and page
tables against a plain loop, and the three run together as a decoding loop."""
import math

import pytest
import torch

import exact_attention_58_gb300 as ea
from paged_ref import check_attention, make_paged, ref_page_table

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def run(x, causal, window=0, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [kw.pop(n, getattr(x, n)) for n in
            ("q", "k_cache", "v_cache", "page_table", "seq_lens", "cu")]
    if kw.pop("wide", False):   # room for 64000 keys and more, unused
        args[3] = torch.nn.functional.pad(args[3], (0, 8000), value=-1)
    args = [a if a.is_cuda else a.cuda() for a in args]
    o, lse = ea.attn_fwd_paged(*args, kw.pop("max_q", x.max_q), causal=causal, window=window,
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
@pytest.mark.parametrize("wide", [False, True], ids=["short table", "wide table"])
def test_lengths_and_heads(lens, d, heads, causal, wide):
    x = make_paged(*lens, *heads, d, 16, seed=d + sum(lens[1]), poison=math.nan)
    check_attention(*run(x, causal, wide=wide), x, causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 24, 48, 64, 128, 256, 384])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [40, 1, 200]], ids=str)
def test_page_sizes(d, page, q_lens):
    x = make_paged(q_lens, [300, 129, 777], 4, 2, d, page, seed=page, poison=math.inf)
    check_attention(*run(x, True), x, True)
    check_attention(*run(x, True, wide=True), x, True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens", [[60] * 8, [1] * 8], ids=str)
def test_last_tile_of_longer_contexts(d, q_lens):
    """The last tile's V rows past the end are cleared only once that tile has
    arrived, however late the pages before it come in."""
    k_lens = [2700, 300, 1111, 129, 255, 2047, 513, 385]
    x = make_paged(q_lens, k_lens, 4, 2, d, 8, seed=d, poison=math.nan)
    for _ in range(5):
        check_attention(*run(x, True), x, True)


@pytest.mark.parametrize("window", [1, 7, 128, 300, 10**6, 2**31 - 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens", [[1, 1], [3, 2], [250, 30]], ids=str)
def test_window(window, causal, q_lens):
    x = make_paged(q_lens, [600, 333], 4, 2, 64, 16, seed=window % 1000, poison=math.nan)
    if causal:
        # pages that the window has left behind are given back
        for b, (n, L) in enumerate(zip(q_lens, [600, 333])):
            gone = max(0, L - n - window + 1) // 16
            lost = x.page_table[b, :gone].long()
            x.k_cache[lost], x.v_cache[lost] = math.nan, math.nan
            x.page_table[b, :gone] = 2**31 - 1
    check_attention(*run(x, causal, window), x, causal, window)
    check_attention(*run(x, causal, window, wide=True), x, causal, window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens", [[1, 1], [9, 1], [160, 2]], ids=str)
def test_fp16(d, q_lens):
    x = make_paged(q_lens, [400, 1300], 6, 2, d, 32, dtype=FP16, seed=d, poison=math.nan)
    check_attention(*run(x, True), x, True)
    check_attention(*run(x, True, wide=True), x, True)


@pytest.mark.parametrize("heads", [(128, 1), (65, 1), (48, 1), (20, 4), (6, 2), (16, 1), (33, 1)],
                         ids=str)
@pytest.mark.parametrize("q_lens", [[1, 1], [2, 1], [11, 40]], ids=str)
def test_groups(heads, q_lens):
    x = make_paged(q_lens, [140, 300], *heads, 64, 16, seed=heads[0], poison=math.nan)
    check_attention(*run(x, True), x, True)
    check_attention(*run(x, True, wide=True), x, True)


def test_spiky_keys():
    """Row maxima that keep growing along the keys: every block rescales."""
    for q_lens in ([1], [50]):
        x = make_paged(q_lens, [1500], 4, 1, 128, 16, seed=5, poison=math.nan)
        ramp = torch.linspace(0.1, 6, 1500)[:, None, None].double()
        k = (x.keys[0] * ramp).to(BF16)
        x.keys[0] = k.double()
        for c in range(-(-1500 // 16)):
            m = min(16, 1500 - 16 * c)
            x.k_cache[x.page_table[0, c], :, :m] = k[16 * c:16 * c + m].transpose(0, 1)
        check_attention(*run(x, True), x, True)
        check_attention(*run(x, True, wide=True), x, True)


def test_many_requests():
    """More requests than threads of a block, most of them short, some empty."""
    g = torch.Generator().manual_seed(3)
    k_lens = torch.randint(0, 300, (700,), generator=g).tolist()
    q_lens = [min(1, n) for n in k_lens]
    x = make_paged(q_lens, k_lens, 2, 1, 64, 16, seed=9, poison=math.nan)
    check_attention(*run(x, True), x, True)
    q_lens = [min(n, i % 5) for i, n in enumerate(k_lens)]
    q_lens[650], k_lens[650] = 333, 400
    x = make_paged(q_lens, k_lens, 2, 1, 64, 16, seed=10, poison=math.nan)
    check_attention(*run(x, True), x, True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 4, 150])
def test_strided_views(q_len, d):
    """Queries as a slice of a fused projection, or heads first; token-major
    pages; K and V side by side in one array."""
    H, Hkv, page = 4, 2, 16
    x = make_paged([q_len, 1], [500, 77], H, Hkv, d, page, seed=q_len, poison=math.nan)
    T = q_len + 1
    fused = torch.full((T, H + 2 * Hkv, d), math.nan, dtype=BF16)
    fused[:, :H] = x.q
    base = run(x, True)
    check_attention(*base, x, True)
    kv = torch.stack([x.k_cache, x.v_cache], 1).cuda()                  # [pages, 2, Hkv, page, d]
    token_major = [t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
                   for t in (x.k_cache, x.v_cache)]
    for kc, vc in ((kv[:, 0], kv[:, 1]), token_major):
        assert not kc.is_contiguous()
        o, lse = run(x, True, q=fused.cuda()[:, :H], k_cache=kc, v_cache=vc)
        assert torch.equal(o, base[0]) and torch.equal(lse, base[1])
    heads_first = x.q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    o, lse = run(x, True, q=heads_first)
    assert o.is_contiguous() and torch.equal(o, base[0]) and torch.equal(lse, base[1])


@pytest.mark.parametrize("q_lens", [[1, 1, 0], [40, 1, 130]], ids=str)
def test_rows_behind_the_last_sequence_are_left(q_lens):
    x = make_paged(q_lens, [200, 5, 400], 4, 2, 64, 16, seed=1, poison=math.nan, extra_rows=37)
    x.q[sum(q_lens):] = math.nan
    out = torch.full(x.q.shape, 7.0, dtype=BF16, device="cuda")
    lse = torch.full((4, x.q.shape[0]), 7.0, device="cuda")
    run(x, True, out=out, lse=lse)
    check_attention(out, lse, x, True)
    T = sum(q_lens)
    assert bool((out[T:] == 7).all()) and bool((lse[:, T:] == 7).all())


@pytest.mark.parametrize("q_len", [1, 3, 90])
def test_max_seqlen_is_only_a_bound(q_len):
    x = make_paged([q_len, 1], [700, 300], 4, 2, 128, 16, seed=2, poison=math.nan)
    run(x, True, max_q=1000)
    check_attention(*run(x, True, max_q=1000), x, True)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_tiles(d):
    """Several rounds of query tiles per CTA: uniform and ragged requests, empty
    ones among them, with and without a window."""
    for q_lens, k_lens in (([130] * 40, [200] * 40),
                           ([0, 300, 1, 77] * 10, [50, 350, 400, 90] * 10)):
        x = make_paged(q_lens, k_lens, 8, 8, d, 16, seed=d, poison=math.nan)
        check_attention(*run(x, True), x, True)
        check_attention(*run(x, False, 60), x, False, 60)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (64, 1), (65, 1)], ids=str)
def test_single_tokens_beside_a_chunk(d, heads):
    """Most requests short beside the longest: they and the long ones go to a
    kernel each, and every row is written once."""
    group = heads[0] // heads[1]
    q_lens = [1] * 14 + [150] + [16 // group, 0, 16 // group + 1, 64 // group + 1] + [2] * 6
    k_lens = [37 * i + q + 5 for i, q in enumerate(q_lens)]
    k_lens[3], k_lens[20] = 0, 1
    x = make_paged(q_lens, k_lens, *heads, d, 16, seed=d, poison=math.nan, extra_rows=3)
    for wide in (False, True):
        out = torch.full(x.q.shape, 7.0, dtype=BF16, device="cuda")
        lse = torch.full((heads[0], x.q.shape[0]), 7.0, device="cuda")
        run(x, True, 90, wide=wide, out=out, lse=lse)
        check_attention(out, lse, x, True, 90)
        assert bool((out[-3:] == 7).all()) and bool((lse[:, -3:] == 7).all())


@pytest.mark.parametrize("longest,max_q", [(200, 200), (2, 200), (0, 200), (2, 2), (0, 2)])
@pytest.mark.parametrize("B", [8, 40])
def test_mostly_empty_batches(longest, max_q, B):
    """Calls with room for more than they hold: few requests have queries, or
    none, whichever kernels the sizes choose."""
    q_lens = ([0, 0, longest] + [0] * 5) * (B // 8)
    rows = sum(q_lens) + 9
    x = make_paged(q_lens, [500 + q for q in q_lens], 4, 2, 64, 16, seed=1, poison=math.nan, extra_rows=9)
    for wide in (False, True):
        out = torch.full((rows, 4, 64), 7.0, dtype=BF16, device="cuda")
        lse = torch.full((4, rows), 7.0, device="cuda")
        run(x, True, max_q=max_q, wide=wide, out=out, lse=lse)
        check_attention(out, lse, x, True)
        assert bool((out[-9:] == 7).all()) and bool((lse[:, -9:] == 7).all())


@pytest.mark.parametrize("q_len", [1, 40])
def test_requests_share_pages(q_len):
    """The same page in several requests: a prompt that they begin with."""
    x = make_paged([q_len] * 3, [400, 400, 400], 4, 2, 128, 16, seed=5, poison=math.nan)
    x.page_table[1:, :20] = x.page_table[0, :20]
    for b in (1, 2):
        x.keys[b][:320], x.values[b][:320] = x.keys[0][:320], x.values[0][:320]
    check_attention(*run(x, True), x, True)


@pytest.mark.parametrize("q_len", [1, 100])
def test_guard_bands(q_len):
    """Nothing is written outside O and LSE, nor beside the caches' slots."""
    x = make_paged([q_len, 1, 7], [300, 90, 40], 4, 2, 64, 16, seed=3, poison=math.nan)
    n = x.q.numel()
    band = 4096
    buf = torch.full((n + 2 * band,), 3.0, dtype=BF16, device="cuda")
    lbuf = torch.full((4 * x.q.shape[0] + 2 * band,), 3.0, device="cuda")
    out = buf[band:band + n].view(x.q.shape)
    lse = lbuf[band:-band].view(4, -1)
    for wide in (False, True):
        run(x, True, out=out, lse=lse, wide=wide)
        check_attention(out, lse, x, True)
        for b in (buf, lbuf):
            assert bool((b[:band] == 3).all()) and bool((b[-band:] == 3).all())


def test_two_streams_at_once():
    """Calls with a workspace each, on two streams at the same time."""
    a = make_paged([1] * 5, [3000, 100, 900, 2000, 50], 8, 2, 128, 16, seed=50)
    b = make_paged([300, 40], [1300, 700], 8, 2, 128, 16, seed=51)
    ref = [run(x, True, wide=True) for x in (a, b)]
    dev = [[t.cuda() for t in (x.q, x.k_cache, x.v_cache,
                               torch.nn.functional.pad(x.page_table, (0, 8000), value=-1),
                               x.seq_lens, x.cu)] for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, x in enumerate((a, b)):
            got[i].append(ea.attn_fwd_paged(*dev[i], x.max_q, causal=True, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, ref[i][0]) and torch.equal(lse, ref[i][1])


def test_scale_and_dirty_workspace():
    """An own scale, and a workspace whose contents on entry are NaN."""
    for q_lens in ([1, 1], [20, 100]):
        x = make_paged(q_lens, [3000, 200], 8, 2, 128, 16, seed=4, poison=math.nan)
        n = ea.attn_fwd_paged_workspace_size(2, 8, 2, sum(q_lens), x.max_q,
                                             x.page_table.shape[1] + 8000, 16, 128)
        assert n > 0
        ws = torch.full((n // 4 + 1,), math.nan, device="cuda")
        check_attention(*run(x, True, scale=0.3, workspace=ws, wide=True), x, True, scale=0.3)


def test_same_result_every_time():
    x = make_paged([1] * 7 + [4], [4000, 33, 800, 1, 129, 2500, 64, 900], 8, 2, 128, 16, seed=8,
                   poison=math.nan)
    for wide in (False, True):
        a = run(x, True, wide=wide)
        for _ in range(3):
            b = run(x, True, wide=wide)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_cache_past_32_bit_offsets():
    """Pages more than 2^31 elements into the pool."""
    page, Hkv, d = 64, 8, 128
    num_pages = 2**31 // (page * Hkv * d) + 50
    x = make_paged([1, 70], [500, 200], 16, Hkv, d, page, seed=6)
    kc = torch.empty(num_pages, Hkv, page, d, dtype=BF16, device="cuda")
    vc = torch.empty_like(kc)
    table = x.page_table.clone()
    used = x.page_table[x.page_table >= 0]
    table[x.page_table >= 0] = used + num_pages - x.k_cache.shape[0]
    for src, dst in zip(used.tolist(), table[x.page_table >= 0].tolist()):
        # written through the cache-append operator
        for h_src, h_dst in ((x.k_cache, kc), (x.v_cache, vc)):
            h_dst[dst].fill_(0)
        slots = torch.arange(dst * page, (dst + 1) * page, dtype=torch.int64, device="cuda")
        ea.attn_cache_append(x.k_cache[src].transpose(0, 1).contiguous().cuda(),
                             x.v_cache[src].transpose(0, 1).contiguous().cuda(), kc, vc, slots)
    check_attention(*run(x, True, k_cache=kc, v_cache=vc, page_table=table), x, True)


def test_long_context():
    """One token over 70001 keys: sampled through the values.  All keys equal
    gives the mean of the values."""
    L, page, d = 70001, 64, 128
    n = -(-L // page)
    kc = torch.ones(n, 2, page, d, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    vc = torch.randn(n, 2, page, d, device="cuda", generator=g).to(BF16)
    table = torch.randperm(n, device="cuda", generator=g).to(torch.int32)[None].contiguous()
    V = vc[table[0].long()].transpose(0, 1).reshape(2, -1, d)[:, :L].double()
    q = torch.ones(1, 8, d, dtype=BF16, device="cuda")
    seq = torch.tensor([L], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    o, lse = ea.attn_fwd_paged(q, kc, vc, table, seq, cu, 1, causal=True)
    ref = V.mean(1).repeat_interleave(4, 0)[None]
    # equal weights: P rounds by the same factor everywhere or not at all, but
    # the bound allows each weight its own rounding
    u = 2.0**-8
    tol = V.abs().mean(1).repeat_interleave(4, 0)[None] * (u + (L + 64) * 2.0**-23) + u * ref.abs()
    assert bool(((o.double() - ref).abs() <= tol * (1 + u)).all())
    z = math.sqrt(d) + math.log(L)
    assert float((lse.double() - z).abs().max()) <= (L + 64) * 2.0**-24 + (d + 8) * 2.0**-24 * 12 + 1e-5


@pytest.mark.parametrize("q_len", [1, 100])
def test_bad_pages_are_reported(q_len):
    x = make_paged([q_len, 1], [400, 300], 4, 2, 64, 16, seed=11)
    for bad in (-5, x.k_cache.shape[0], 2**31 - 1):
        table = x.page_table.clone()
        table[1, 3] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = ea.attn_fwd_paged(x.q.cuda(), x.k_cache.cuda(), x.v_cache.cuda(), table.cuda(),
                                   x.seq_lens.cuda(), x.cu.cuda(), x.max_q, causal=True,
                                   dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 1
        # the other request is not touched by it
        ref, _ = run(x, True)
        assert torch.equal(o[:q_len], ref[:q_len])


@pytest.mark.parametrize("cu,seq", [
    ([0, 3, 2], [50, 60]), ([0, 1, 99], [50, 60]), ([-4, 1, 2], [50, 60]),
    ([0, 1, 2], [-1, 60]), ([0, 1, 2], [50, 1 << 30]), ([0, 30, 31], [50, 60]),
], ids=str)
def test_bad_lengths_are_clamped_and_reported(cu, seq):
    x = make_paged([20, 11], [50, 60], 4, 2, 64, 16, seed=12)
    for max_q in (1, 20):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ea.attn_fwd_paged(x.q.cuda(), x.k_cache.cuda(), x.v_cache.cuda(), x.page_table.cuda(),
                          torch.tensor(seq, dtype=torch.int32, device="cuda"),
                          torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q, causal=True,
                          dev_status=status)
        torch.cuda.synchronize()
        if max_q == 1 or cu != [0, 30, 31]:
            assert int(status.item()) == 1


def test_other_stream_and_graph_with_new_lengths():
    """A captured call, replayed after the lengths, tables and queries changed
    in place, gives what a fresh call gives; also on a stream of its own."""
    H, Hkv, d, page = 8, 2, 128, 16
    for q_len in (1, 80):
        a = make_paged([q_len] * 3, [500, 900, 90], H, Hkv, d, page, seed=20)
        b = make_paged([q_len] * 3, [130, 80, 1000], H, Hkv, d, page, seed=21)
        pages = max(a.k_cache.shape[0], b.k_cache.shape[0])
        width = max(a.page_table.shape[1], b.page_table.shape[1])

        def load(x, bufs):
            for name, t in bufs.items():
                src = getattr(x, name)
                t[tuple(slice(0, n) for n in src.shape)].copy_(src)

        bufs = dict(q=torch.zeros_like(a.q, device="cuda"),
                    k_cache=torch.zeros(pages, Hkv, page, d, dtype=BF16, device="cuda"),
                    v_cache=torch.zeros(pages, Hkv, page, d, dtype=BF16, device="cuda"),
                    page_table=torch.zeros(3, width, dtype=torch.int32, device="cuda"),
                    seq_lens=torch.zeros(3, dtype=torch.int32, device="cuda"),
                    cu=torch.zeros(4, dtype=torch.int32, device="cuda"))
        load(a, bufs)
        out = torch.zeros_like(bufs["q"])
        lse = torch.zeros(H, a.q.shape[0], device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())

        def call(**kw):
            ea.attn_fwd_paged(*(bufs[n] for n in ("q", "k_cache", "v_cache", "page_table",
                                                  "seq_lens", "cu")),
                              q_len, causal=True, out=out, lse=lse, **kw)

        call(stream=side)
        side.synchronize()
        check_attention(out, lse, a, True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        load(b, bufs)
        graph.replay()
        torch.cuda.synchronize()
        check_attention(out, lse, b, True)


def test_both_ways_into_the_library_agree():
    """The short way through the extension (no stream argument) and the long one
    through ctypes: same results, outputs given or not; and the same refusals."""
    x = make_paged([3, 40, 0, 1], [200, 90, 5, 700], 8, 2, 64, 16, seed=40, poison=math.nan)
    here = torch.cuda.current_stream()
    a = run(x, True, window=100)
    out, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    for kw in (dict(stream=here), dict(stream=here.cuda_stream or 0), dict(out=out, lse=lse),
               dict(workspace=torch.empty(100 << 20, dtype=torch.uint8, device="cuda"), scale=0.125)):
        b = run(x, True, window=100, **kw)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert run(x, True, out=out, lse=lse)[0] is out
    dev = [t.cuda() for t in (x.q, x.k_cache, x.v_cache, x.page_table, x.seq_lens, x.cu)]
    for stream in (None, here):
        for i, bad in ((0, dev[0].float()), (1, dev[1][:, :1]), (3, dev[3].long()), (4, dev[4][:1]),
                       (5, x.cu), (0, dev[0][:, :, ::2])):
            with pytest.raises(ValueError):
                ea.attn_fwd_paged(*dev[:i], bad, *dev[i + 1:], 40, stream=stream)
        for kw, status in ((dict(scale=-1.0), 1), (dict(workspace=torch.empty(4, device="cuda")), 4)):
            wide = torch.nn.functional.pad(dev[3], (0, 8000), value=-1)
            with pytest.raises(ea.AttnError) as e:
                ea.attn_fwd_paged(*dev[:3], wide, *dev[4:], 40, stream=stream, **kw)
            assert e.value.status == status
        with pytest.raises(ValueError):
            ea.attn_fwd_paged(*dev, 40, out=out.float(), stream=stream)
        with pytest.raises(ValueError):
            ea.attn_cache_append(dev[0][:, :2], dev[0][:, :2], dev[1], dev[2],
                                 torch.zeros(3, dtype=torch.int64, device="cuda"), stream=stream)
        with pytest.raises(ea.AttnError) as e:   # an output inside an input
            ea.attn_page_table(dev[4], dev[4], dev[3], dev[5], dev[4][:1], 16, 8, seq_lens=dev[4],
                               stream=stream)
        assert e.value.status == 1


# ---------------------------------------------------------------------------
# cache append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,Hkv,d,page", [(1, 1, 64, 8), (7, 3, 128, 16), (300, 8, 128, 48),
                                          (65, 2, 256, 64)])
def test_append(dtype, T, Hkv, d, page):
    g = torch.Generator().manual_seed(T)
    pages = T // page + 5
    kc = torch.randn(pages, Hkv, page, d, generator=g).to(dtype)
    vc = torch.randn(pages, Hkv, page, d, generator=g).to(dtype)
    qkv = torch.randn(T, 3 * Hkv, d, generator=g).to(dtype)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int64)
    slots[::5] = -1
    ref_k, ref_v = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            ref_k[s // page, :, s % page] = qkv[t, Hkv:2 * Hkv]
            ref_v[s // page, :, s % page] = qkv[t, 2 * Hkv:]
    dev = qkv.cuda()
    for k, v in ((dev[:, Hkv:2 * Hkv], dev[:, 2 * Hkv:]),
                 (dev[:, Hkv:2 * Hkv].contiguous(), dev[:, 2 * Hkv:].contiguous())):
        a, b = kc.cuda(), vc.cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ea.attn_cache_append(k, v, a, b, slots.cuda(), dev_status=status)
        assert torch.equal(a.cpu(), ref_k) and torch.equal(b.cpu(), ref_v)
        assert int(status.item()) == 0
    # token-major views of one array
    both = torch.stack([kc, vc], 1).transpose(2, 3).contiguous().cuda().transpose(2, 3)
    ea.attn_cache_append(dev[:, Hkv:2 * Hkv], dev[:, 2 * Hkv:], both[:, 0], both[:, 1], slots.cuda())
    assert torch.equal(both[:, 0].cpu(), ref_k) and torch.equal(both[:, 1].cpu(), ref_v)


def test_append_out_of_range_slots_are_skipped_and_reported():
    kc = torch.zeros(4, 2, 16, 64, dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.ones(3, 2, 64, dtype=BF16, device="cuda")
    for bad in (-2, 64, 2**40, -2**40):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        slots = torch.tensor([5, bad, 6], dtype=torch.int64, device="cuda")
        ea.attn_cache_append(k, k, kc, vc, slots, dev_status=status)
        assert int(status.item()) == 1
        assert float(kc.float().sum()) == 2 * 2 * 64 and float(vc.float().sum()) == 2 * 2 * 64


# ---------------------------------------------------------------------------
# page table
# ---------------------------------------------------------------------------
def make_table(cached, new, page, seed, extra=3, width_extra=2):
    g = torch.Generator().manual_seed(seed)
    held = [-(-c // page) for c in cached]
    width = max(-(-(c + n) // page) for c, n in zip(cached, new)) + width_extra
    need = sum(-(-(c + n) // page) for c, n in zip(cached, new)) - sum(held)
    order = torch.randperm(sum(held) + need + extra, generator=g).tolist()
    table = [[-7] * width for _ in cached]
    for b, h in enumerate(held):
        for c in range(h):
            table[b][c] = order.pop()
    return table, order, need


def run_table(cached, new, table, free, num_free, page, max_tokens, **kw):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = i32(table)
    cu, seq, slots, taken = ea.attn_page_table(i32(cached), i32(new), t, i32(free), i32([num_free]),
                                               page, max_tokens, dev_status=status, **kw)
    return (cu.tolist(), seq.tolist(), slots.tolist(), int(taken.item()), t.tolist()), int(status.item())


@pytest.mark.parametrize("B,q_hi,ctx_hi,page,pad", [
    (1, 1, 0, 16, 0), (1, 1, 100, 8, 5), (5, 1, 64, 16, 0), (40, 30, 200, 16, 100),
    (513, 3, 90, 48, 1), (1500, 2, 40, 16, 700), (3, 2500, 3000, 64, 0), (17, 0, 50, 16, 9)])
def test_page_table(B, q_hi, ctx_hi, page, pad):
    g = torch.Generator().manual_seed(B + q_hi)
    new = torch.randint(0, q_hi + 1, (B,), generator=g).tolist()
    if B == 1:
        new = [max(1, q_hi)]
    cached = torch.randint(0, ctx_hi + 1, (B,), generator=g).tolist()
    cached[::3] = [c // page * page for c in cached[::3]]   # full last pages
    table, free, _ = make_table(cached, new, page, seed=B)
    T = max(1, sum(new) + pad)
    got, status = run_table(cached, new, table, free + [12345], len(free), page, T)
    assert got == ref_page_table(cached, new, table, free, len(free), page, T)
    assert status == 0


def test_page_table_runs_out_of_pages():
    cached, new, page = [10, 30, 16], [40, 1, 33], 16
    table, free, need = make_table(cached, new, page, seed=1)
    got, status = run_table(cached, new, table, free, need - 2, page, 80)
    assert got == ref_page_table(cached, new, table, free, need - 2, page, 80)
    assert status == 1 and -1 in got[2][:74]


@pytest.mark.parametrize("cached,new,num_free,tokens", [
    ([-3, 5], [1, 1], 4, 4), ([3, 5], [-1, 1], 4, 4), ([3, 5], [200, 1], 4, 300),
    ([3, 5], [2, 9], 4, 4), ([3, 5], [1, 1], 99, 4), ([3, 5], [1, 1], -1, 4),
    ([2**31 - 1, 5], [2**31 - 1, 1], 4, 4)], ids=str)
def test_page_table_bad_values_are_clamped_and_reported(cached, new, num_free, tokens):
    page, width = 8, 4
    table = [[0, 1, 2, 3], [4, 5, 6, 7]]
    got, status = run_table(cached, new, table, [8, 9, 10, 11, 12], num_free, page, tokens)
    assert status == 1
    cu, seq, slots, taken, _ = got
    assert len(slots) == tokens and all(s == -1 or 0 <= s < 13 * page for s in slots)
    assert 0 <= cu[1] <= cu[2] <= tokens and all(0 <= s <= page * width for s in seq)
    assert 0 <= taken <= 5


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_serving_loop():
    """Prompts, then single and drafted tokens, through tables, cache and
    attention; every step against the definition on the whole history."""
    H, Hkv, d, page, B, width = 8, 2, 128, 16, 5, 40
    g = torch.Generator().manual_seed(7)
    pool = 130
    kc = torch.full((pool, Hkv, page, d), math.nan, dtype=BF16, device="cuda")
    vc = torch.full_like(kc, math.nan)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pool, generator=g).to(torch.int32).cuda()
    num_free = torch.tensor([pool], dtype=torch.int32, device="cuda")
    cached = torch.zeros(B, dtype=torch.int32, device="cuda")
    keys = [torch.zeros(0, Hkv, d, dtype=torch.float64) for _ in range(B)]
    values = [t.clone() for t in keys]
    steps = [[200, 17, 0, 128, 1], [1, 1, 90, 1, 1], [1, 1, 1, 1, 1], [4, 1, 4, 0, 2], [1, 1, 1, 1, 1],
             [0, 16, 0, 111, 33]]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step, new in enumerate(steps):
        T = sum(new)
        q, k, v = (torch.randn(T, n, d, generator=g).to(BF16) for n in (H, Hkv, Hkv))
        lens = torch.tensor(new, dtype=torch.int32, device="cuda")
        cu, seq, slots, taken = ea.attn_page_table(cached, lens, table, free, num_free, page, T + 3,
                                                   dev_status=status)
        ea.attn_cache_append(k.cuda(), v.cuda(), kc, vc, slots[:T], dev_status=status)
        o, lse = ea.attn_fwd_paged(q.cuda(), kc, vc, table, seq, cu, max(new), causal=True,
                                   dev_status=status)
        num_free -= taken
        cached = seq
        t = 0
        for b, n in enumerate(new):
            keys[b] = torch.cat([keys[b], k[t:t + n].double()])
            values[b] = torch.cat([values[b], v[t:t + n].double()])
            t += n
        x = make_paged([1], [1], H, Hkv, d, page)
        x.q, x.cu, x.keys, x.values = q, cu.cpu(), keys, values
        check_attention(o, lse, x, True)
    assert int(status.item()) == 0
    assert int(num_free.item()) == pool - sum(-(-t.shape[0] // page) for t in keys)


def test_agrees_with_packed_attention():
    """Whole prompts through the cache give attn_fwd_varlen's results to within
    the rounding of both."""
    H, d, page = 4, 128, 16
    lens = [300, 77, 128]
    x = make_paged(lens, lens, H, H, d, page, seed=30)
    o, lse = run(x, True)
    check_attention(o, lse, x, True)
    k = torch.cat(x.keys).to(BF16).cuda()
    v = torch.cat(x.values).to(BF16).cuda()
    o2, lse2 = ea.attn_fwd_varlen(x.q.cuda(), k, v, x.cu.cuda(), x.cu.cuda(), 300, 300, causal=True)
    check_attention(o2, lse2, x, True)
