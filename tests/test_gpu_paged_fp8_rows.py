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


# single tokens; chunks that clusters share, and CTAs of a second launch's join; several
# rounds of tiles a CTA
SHAPES = [([1, 2], [300, 77]), ([70, 40], [300, 530]), ([300], [1500]), ([130] * 40, [200] * 40)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0][:2]}x{len(s[0])}")
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("size", [0.0, 2.0**-110])
@pytest.mark.parametrize("k_scale", [0.0, 2.0**-48, 2.0**-34])
def test_queries_of_nothing_over_keys_of_nothing(shape, d, size, k_scale):
    """Zero (or next to zero) queries over a cache of zero keys, as in a warm-up step: every
    key weighs the same, O is the mean of V and LSE the logarithm of their number."""
    x = make_fp8(*shape, 4, 4 if len(shape[0]) > 2 else 2, d, 16, seed=d)
    x.q = torch.full_like(x.q, size)
    x.k_cache = torch.zeros_like(x.k_cache.view(torch.uint8)).view(torch.float8_e4m3fn)
    x.k_scale.fill_(k_scale)
    for k in x.keys:
        k.zero_()
    for wide in (False, True):
        check_rows(*run(x, True, wide=wide), x, True)
        check_rows(*run(x, False, 60, wide=wide), x, False, 60)


@pytest.mark.parametrize("scale", [2.0**-110, 2.0**100])
@pytest.mark.parametrize("q_len", [1, 70])
def test_softmax_scales_far_from_one(scale, q_len):
    """The factor of the scores leaves fp32's range on either side, over keys of nothing."""
    x = make_fp8([q_len], [300], 4, 2, 64, 16, seed=1)
    x.k_cache = torch.zeros_like(x.k_cache.view(torch.uint8)).view(torch.float8_e4m3fn)
    x.k_scale.fill_(2.0**-48 if scale < 1 else 2.0**40)
    x.keys[0].zero_()
    check_rows(*run(x, True, scale=scale), x, True, scale=scale)
