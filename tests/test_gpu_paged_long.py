"""Paged attention over long contexts on the GPU, against the definition in 64
bits with an error bound per element."""
import dataclasses
import math

import pytest
import torch

import exact_attention_58_gb300 as ea
from paged_ref import (FP16_LEAST, check_attention, heavy_tail, make_paged, ref_attention,
                       spread_keys)

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def run(x, causal=True, window=0, *, width=0, max_q=None):
    """The operator on x, its page table widened to `width` columns."""
    table = x.page_table
    if width > table.shape[1]:
        table = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = ea.attn_fwd_paged(*(t.cuda() for t in (x.q, x.k_cache, x.v_cache, table, x.seq_lens, x.cu)),
                               x.max_q if max_q is None else max_q, causal=causal, window=window,
                               dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0, f"device status {int(status.item())}"
    return o, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,heads,L", [
    (1, 4, 70001),     # decode kernel, pieces joined by a second launch
    (1, 2, 1500),      # decode kernel, a cluster
    (5, 8, 20000),     # two softmax groups
    (70, 2, 20000),    # tile kernel, shared out
    (300, 2, 3000),
], ids=str)
def test_fp16_tail_is_not_lost(n, heads, L, d):
    """Weights 2^-25 of the largest and below, which fp16 would hold as zero, count
    in O as they do in the sum that O is divided by."""
    x = heavy_tail(n, L, heads, d, 64, 17.6, seed=d)
    check_attention(*run(x), x, True, least=FP16_LEAST)


def on_gpu(x):
    """The reference's own keys and values on the GPU: it computes there."""
    return dataclasses.replace(x, keys=[t.cuda() for t in x.keys], values=[t.cuda() for t in x.values])


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (256, BF16), (64, FP16), (128, FP16)], ids=str)
@pytest.mark.parametrize("n,H,Hkv,L", [
    (1, 16, 1, 70001),      # one key head: 152 pieces a row, two batches of the join's eight warps
    (1, 16, 2, 70001),
    (1, 32, 1, 131072),     # two softmax groups
    (4, 16, 1, 131072),     # 64 rows
    (60, 4, 1, 70001),      # tile kernel: 76 pieces and more a tile, joined by a launch
    (150, 16, 4, 20000),    # a cluster a tile
    (700, 32, 8, 9000),     # a CTA a tile
], ids=str)
def test_long_contexts(n, H, Hkv, L, d, dtype):
    """Random keys; every 128 of them hold one that counts in some row."""
    x = on_gpu(spread_keys(n, L, H, Hkv, d, 64, seed=d + n, dtype=dtype))
    check_attention(*run(x), x, True, least=FP16_LEAST if dtype == FP16 else None)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("few", [[1] * 15, [1, 4, 0, 5, 2, 1, 1, 1, 3, 1, 1, 1, 4, 1, 1]], ids=str)
def test_single_tokens_beside_a_long_prompt(d, few):
    """Two launches, of which the tile kernel's is the persistent one: more tiles
    than SMs, most of them of no request."""
    q_lens = few[:7] + [2000] + few[7:]
    k_lens = [2500 if n == 2000 else 150 * i + n for i, n in enumerate(q_lens)]
    x = make_paged(q_lens, k_lens, 32, 8, d, 16, seed=d, poison=math.nan, extra_rows=5)
    x = on_gpu(x)
    for width in (0, 600):   # 9600 keys: two launches
        check_attention(*run(x, width=width), x, True)
        check_attention(*run(x, window=300, width=width), x, True, 300)


def test_work_past_2_to_24_key_blocks():
    """4096 requests that share their pages: 2^24 key blocks over all heads, where
    a CTA's run and the pieces of a tile are counted in 64 bits."""
    kinds, B, H, d, page = 8, 4096, 8, 64, 64
    lens = [65536 + 128 * i + 17 * (i % 3) for i in range(kinds)]
    one = spread_keys(1, max(lens), H, H, d, page, seed=1)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(kinds, H, d, generator=g).to(BF16)
    q[0] = one.q[0]
    x = dataclasses.replace(one, q=q, seq_lens=torch.tensor(lens, dtype=torch.int32),
                            cu=torch.arange(kinds + 1, dtype=torch.int32),
                            page_table=one.page_table.repeat(kinds, 1).contiguous(),
                            keys=[one.keys[0][:n] for n in lens], values=[one.values[0][:n] for n in lens])
    O, lse, tol, lse_tol = ref_attention(on_gpu(x), True)
    big = dataclasses.replace(x, q=q.repeat(B // kinds, 1, 1), seq_lens=x.seq_lens.repeat(B // kinds),
                              cu=torch.arange(B + 1, dtype=torch.int32),
                              page_table=x.page_table.repeat(B // kinds, 1).contiguous())
    assert sum(-(-n // 128) for n in lens) * (B // kinds) * H >= 1 << 24
    o, z = run(big)
    n = B // kinds
    assert bool(((o.double() - O.repeat(n, 1, 1)).abs() <= tol.repeat(n, 1, 1)).all())
    assert bool(((z.double() - lse.repeat(1, n)).abs() <= lse_tol.repeat(1, n)).all())
