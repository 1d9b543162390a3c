"""Rotary positions and the 8-bit cache on a stream given by name, and beside the
ordinary cache: same results, in the order of the given stream."""
import pytest
import torch

import exact_attention_58_gb300 as ea

pytestmark = pytest.mark.gpu


def rows(*shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_step_on_a_given_stream(dtype):
    """Every call of a step with stream=, its inputs written on that stream just
    before, behind work that keeps the stream busy."""
    H, Hkv, d, page, cached, new = 6, 2, 64, 16, [0, 9, 70, 16], [5, 1, 20, 3]
    T = sum(new)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((4, 8), -1, dtype=torch.int32, device="cuda")
    table[1, :1], table[2, :5], table[3, :1] = i32([30]), i32([7, 3, 11, 2, 20]), i32([5])
    free = i32([12, 13, 14, 15])
    cu, lens, slots, _ = ea.attn_page_table(i32(cached), i32(new), table, free, i32([4]), page, T)
    assert bool((slots >= 0).all())
    f = ea.attn_rope_frequencies(d, device="cuda")[0]
    q, k, v = (rows(T, n, d, dtype=dtype, seed=i) for i, n in enumerate((H, Hkv, Hkv)))
    dense = rows(2, H, 50, d, dtype=dtype, seed=9)
    old = [rows(32, Hkv, page, d, dtype=dtype, seed=s) for s in (4, 5)]
    at = torch.arange(32 * page, dtype=torch.int64, device="cuda")

    def caches():
        c8 = [torch.zeros(32, Hkv, page, d, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        sc = [torch.ones(32, Hkv, device="cuda") for _ in range(2)]
        flat = [o.transpose(1, 2).reshape(32 * page, Hkv, d) for o in old]
        ea.attn_cache_append_fp8(*flat, *c8, *sc, at)
        return [o.clone() for o in old], c8, sc

    def step(x, c16, c8, sc, **kw):
        y, _ = ea.attn_rope(x, None, f, **kw)
        qr = ea.attn_cache_append_rope(q, k, v, *c16, slots, f, cu_seqlens_q=cu, seq_lens=lens, **kw)
        ea.attn_cache_append_fp8(k, v, *c8, *sc, slots, **kw)
        o, lse = ea.attn_fwd_paged_fp8(qr, *c8, *sc, table, lens, cu, max(new), causal=True, **kw)
        return [y, qr, o, lse, *c16, *(c.view(torch.uint8) for c in c8), *sc]

    want = step(dense, *caches())
    mine = caches()
    stream = torch.cuda.Stream()
    late = torch.zeros_like(dense)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        a = torch.randn(2048, 2048, device="cuda")
        for _ in range(20):
            a = a @ a * 1e-3
        late.copy_(dense)
    got = step(late, *mine, stream=stream)   # not the current stream
    stream.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
