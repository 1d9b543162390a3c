"""The long-context tests' references and bounds on the CPU: that they see what
they are for."""
import dataclasses
import math

import pytest
import torch

from paged_ref import FP16_LEAST, check_attention, heavy_tail, ref_attention, spread_keys


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


@pytest.mark.parametrize("n,H,L", [(1, 16, 70001), (1, 32, 131072), (4, 16, 131072), (60, 2, 70001)])
def test_long_context_mistakes_are_seen(n, H, L):
    """One block of 128 keys lost, wherever it is; two blocks' values in one
    another's place; a piece of the keys left out."""
    x = spread_keys(n, L, H, 1, 64, 64, seed=3)
    O, lse, _, _ = ref_attention(x, True)
    check_attention(O, lse, x, True)
    K, V = x.keys[0], x.values[0]

    def seen(k, v):
        o, z, _, _ = ref_attention(dataclasses.replace(x, keys=[k], values=[v]), True)
        with pytest.raises(AssertionError):
            check_attention(o, z, x, True)

    for j in (0, 77, L // 128 - 5):
        keep = torch.ones(L, dtype=torch.bool)
        keep[128 * j:128 * j + 128] = False
        seen(K[keep], V[keep])
    for a, b in ((0, 1), (100, 400)):
        swapped = V.clone()
        swapped[128 * a:128 * a + 128], swapped[128 * b:128 * b + 128] = (
            V[128 * b:128 * b + 128], V[128 * a:128 * a + 128])
        seen(K, swapped)
    piece = L // 152
    keep = torch.ones(L, dtype=torch.bool)
    keep[40 * piece:41 * piece] = False
    seen(K[keep], V[keep])
