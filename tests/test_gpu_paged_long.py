"""Paged attention over long contexts on the GPU, against the definition in 64
bits with an error bound per element."""
import math

import pytest
import torch

import exact_attention_58_gb300 as ea
from paged_ref import FP16_LEAST, check_attention, heavy_tail

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
