"""The bound per row for attention over the 8-bit cache (CPU): it passes the definition's own
roundings and refuses planted mistakes of single rows, heads and pages."""
import math

import pytest
import torch

from fp8_rows_ref import check_rows, rescale_pages, row_bound
from paged_ref import ref_attention
from rope_fp8_ref import make_fp8


def rounded(x, causal, window=0):
    O, L, _, _ = ref_attention(x, causal, window)
    return O.to(x.q.dtype), L


def sized(d):
    """Query rows of sizes 2^-70 to 2^40, the heads' scales to match."""
    x = make_fp8([3], [300], 6, 2, d, 16, seed=d, poison=False)
    x.k_scale[:, 0] *= 2.0**-38
    x.keys[0][:, 0] *= 2.0**-38
    x.q[:, 0] *= 2.0**38
    x.q[:, 1] *= 2.0**33
    x.q[:, 2] *= 2.0**40
    x.q[:, 3] = 0.0
    x.q[:, 4, 0] = 2.0**6
    x.q[:, 5] *= 2.0**-70
    x.q[:, 5, 1] = 1.0
    return x


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("row", [None, 0, 1, 2, 4, 5])
def test_a_row_turned_by_one_power_too_many(d, row):
    """One head's queries twice as large as they are: refused, whatever the others' sizes."""
    x, y = sized(d), sized(d)
    if row is None:
        check_rows(*rounded(y, True), x, True)
        return
    y.q[1, row] *= 2.0
    with pytest.raises(AssertionError):
        check_rows(*rounded(y, True), x, True)


def test_rows_of_two_heads_changed_places():
    x, y = sized(64), sized(64)
    y.q[:, [4, 5]] = y.q[:, [5, 4]]
    with pytest.raises(AssertionError):
        check_rows(*rounded(y, True), x, True)


@pytest.mark.parametrize("which", ["k", "v"])
def test_a_page_lost_beside_a_large_one(which):
    """The page before one of 2^30 times its size read as zero: refused for the rows that
    attend only the former, and the bound of those does not know of the latter."""
    far = dict(k_pow=30) if which == "k" else dict(v_pow=30)
    x = rescale_pages(make_fp8([40], [64], 2, 1, 64, 16, seed=1, poison=False), 0, [3], **far)
    check_rows(*rounded(x, True), x, True)
    plain = make_fp8([40], [64], 2, 1, 64, 16, seed=1, poison=False)
    before = slice(0, 24)   # queries at keys 24 .. 47, the page starts at 48
    for a, b in zip(row_bound(x, True), row_bound(plain, True)):
        rows = (before,) if a.dim() == 3 else (slice(None), before)
        assert torch.equal(a[rows], b[rows])
    y = rescale_pages(make_fp8([40], [64], 2, 1, 64, 16, seed=1, poison=False), 0, [3], **far)
    (y.keys if which == "k" else y.values)[0][32:48] = 0.0
    with pytest.raises(AssertionError):
        check_rows(*rounded(y, True), x, True)


def test_nan_is_refused():
    x = make_fp8([4], [20], 2, 1, 64, 16, poison=False)
    o, lse = rounded(x, True)
    o[2, 1, 5] = math.nan
    with pytest.raises(AssertionError):
        check_rows(o, lse, x, True)
