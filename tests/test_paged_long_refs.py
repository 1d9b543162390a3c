"""The long-context tests' references and bounds on the CPU: that they see what
they are for."""
import math

import pytest
import torch

from paged_ref import FP16_LEAST, check_attention, heavy_tail, ref_attention


def with_fp16_weights(x, shift):
    """O and LSE of a kernel whose weights are rounded to fp16 for the product with
    V, 2^shift times what they are against the row's largest."""
    O, lse, _, _ = ref_attention(x, True)
    n, heads, d = x.q.shape
    K, V = x.keys[0][:, 0], x.values[0][:, 0]
    p = torch.arange(n)[:, None] + K.shape[0] - n
    for h in range(heads):
        S = (x.q[:, h].double() @ K.T / math.sqrt(d)).masked_fill(torch.arange(K.shape[0]) > p, -math.inf)
        P = torch.exp2((S - S.amax(1, keepdim=True)) / math.log(2) + shift)
        O[:, h] = (P.half().double() @ V) / P.sum(1, keepdim=True)
    return O.half(), lse


@pytest.mark.parametrize("n,L", [(1, 70001), (70, 20000), (1, 1500), (5, 20000), (300, 3000)])
def test_weights_lost_to_fp16_are_seen(n, L):
    x = heavy_tail(n, L, 2, 64, 64, 17.6)
    check_attention(*with_fp16_weights(x, 7), x, True, least=FP16_LEAST)
    with pytest.raises(AssertionError):
        check_attention(*with_fp16_weights(x, 0), x, True, least=FP16_LEAST)
