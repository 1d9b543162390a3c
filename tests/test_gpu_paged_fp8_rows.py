"""Attention over the 8-bit cache on the GPU, each row within a bound of its own
(fp8_rows_ref.py): sizes of queries, keys and values far from one another."""
import math

import pytest
import torch

from fp8_rows_ref import check_rows, rescale_pages
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


# ---------------------------------------------------------------------------
# pages of unlike size side by side
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("shape", SHAPES[1:], ids=lambda s: f"{s[0][:2]}x{len(s[0])}")
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("power", [6, 16, 30, 44])
def test_a_large_page_at_the_end(shape, d, which, power):
    """The last page is 2^power times as large as the others: queries before it do not
    attend it, and see nothing of it."""
    x = make_fp8(*shape, 4, 4 if len(shape[0]) > 2 else 2, d, 16, seed=d + power)
    kw = dict(k_pow=power if which != "v" else 0, v_pow=power if which != "k" else 0)
    for b, L in enumerate(shape[1]):
        rescale_pages(x, b, [(L - 1) // 16], **kw)
    for wide in (False, True):
        check_rows(*run(x, True, wide=wide), x, True)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("page,d", [(8, 64), (24, 64), (64, 64), (128, 64), (16, 128), (24, 256), (64, 256)])
@pytest.mark.parametrize("q_lens", [[1, 4], [150, 33]], ids=str)
def test_pages_of_any_size_in_any_order(dtype, page, d, q_lens):
    """Keys and values of every page at a power of two of its own, 2^-30 to 2^10 (keys
    of large pages point where the queries do not)."""
    x = make_fp8(q_lens, [700, 301], 4, 2, d, page, dtype=dtype, seed=page)
    g = torch.Generator().manual_seed(page)
    for b, L in enumerate([700, 301]):
        for c in range(-(-L // page)):
            rescale_pages(x, b, [c], *torch.randint(-30, 11, (2,), generator=g).tolist(), heads=c % 2)
            rescale_pages(x, b, [c], *torch.randint(-30, 2, (2,), generator=g).tolist(), heads=1 - c % 2)
    for wide in (False, True):
        check_rows(*run(x, True, wide=wide), x, True)
        check_rows(*run(x, True, 50, wide=wide), x, True, 50)
        check_rows(*run(x, False, wide=wide), x, False)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_an_infinite_value_of_a_later_token(d):
    """What the append makes of an infinity (its page's scale is 2^48) is nothing to the
    tokens before it."""
    import exact_attention_58_gb300 as ea
    x = make_fp8([100], [100], 4, 2, d, 16, seed=d, poison=False)
    quiet = run(x, True)
    rows = [torch.full((1, 2, d), s, dtype=BF16, device="cuda") for s in (1.0, math.inf)]
    caches = [t.cuda() for t in (x.k_cache, x.v_cache, x.k_scale, x.v_scale)]
    slot = torch.tensor([int(x.page_table[0, 6]) * 16 + 3], device="cuda")   # the last token, 99
    ea.attn_cache_append_fp8(*rows, *caches, slot)
    assert float(caches[3][int(x.page_table[0, 6]), 0]) == 2.0**48
    got = run(x, True, k_cache=caches[0], v_cache=caches[1], k_scale=caches[2], v_scale=caches[3])
    # tokens of the pages before the last see the same keys and values as without it
    for a, b, dim in ((got[0], quiet[0], 0), (got[1], quiet[1], 1)):
        before = a.narrow(dim, 0, 96).double(), b.narrow(dim, 0, 96).double()
        # (both within the bound of the same row)
        assert bool(((before[0] - before[1]).abs() <= 2.0**-7 * (1 + before[1].abs())).all())


@pytest.mark.parametrize("q_lens", [[1], [3], [60], [200]], ids=str)
def test_a_small_weight_on_large_values(q_lens):
    """A key that outweighs the others with small values, and keys of next to no weight
    with values that make up for it: both halves of O count."""
    x = make_fp8(q_lens, [256], 4, 1, 128, 16, seed=9, poison=False)
    rescale_pages(x, 0, [0, 1, 5], v_pow=-20)
    rescale_pages(x, 0, [2, 9], v_pow=20, k_pow=-3)
    rescale_pages(x, 0, [4], v_pow=-45)
    for wide in (False, True):
        check_rows(*run(x, True, wide=wide), x, True)
