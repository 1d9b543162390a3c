"""Attention over the 8-bit cache on the GPU, each row within a bound of its own
(fp8_rows_ref.py): sizes of queries, keys and values far from one another."""
import pytest
import torch

from fp8_rows_ref import check_rows
from rope_fp8_ref import make_fp8
from test_gpu_paged_fp8 import run

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 3, 70])
def test_queries_of_any_size(d, q_len):
    """bf16 queries far outside fp16's range over keys as far on the other side, rows of
    zeros, rows with one large element: all in one call, each to its own accuracy."""
    x = make_fp8([q_len], [300], 6, 2, d, 16, seed=d)
    x.k_scale[:, 0] *= 2.0**-38
    x.keys[0][:, 0] *= 2.0**-38
    x.q[:, 0] *= 2.0**38
    x.q[:, 1] *= 2.0**33
    x.q[:, 2] *= 2.0**40
    x.q[:, 3] = 0.0
    x.q[:, 4, 0] = 2.0**6
    x.q[:, 5] *= 2.0**-70
    x.q[:, 5, 1] = 1.0
    for wide in (False, True):
        check_rows(*run(x, True, wide=wide), x, True)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("q_lens,k_lens", [([1, 3], [300, 77]), ([70, 1], [300, 77]), ([700], [1500])], ids=str)
def test_rows_of_ordinary_inputs(dtype, q_lens, k_lens):
    x = make_fp8(q_lens, k_lens, 4, 2, 128, 16, dtype=dtype, seed=2, spread=2)
    for wide in (False, True):
        check_rows(*run(x, True, wide=wide), x, True)
        check_rows(*run(x, False, 90, wide=wide), x, False, 90)
