"""Writing into the 8-bit cache: the runs that a page's tokens make, tokens without a slot
among them, bit for bit against a plain loop, and second runs of a page left out."""
import pytest
import torch

import exact_attention_58_gb300 as ea
from rope_fp8_ref import ref_append_fp8

gpu = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def left_out(slots, page, pages):
    """Tokens of second runs: behind a token of their page, or behind tokens without a
    slot, as many as rows at most, that are behind one."""
    inside = lambda s: 0 <= s < page * pages  # noqa: E731
    gone = set()
    for t, s in enumerate(slots):
        if not inside(s):
            continue
        row = s % page
        if t and row and slots[t - 1] == s - 1:
            if t - 1 in gone:
                gone.add(t)
            continue
        for u in range(t - 1, max(-1, t - 1 - max(1, row)), -1):
            if inside(slots[u]):
                if slots[u] // page == s // page:
                    gone.add(t)
                break
    return gone


def append_and_check(calls, Hkv, d, page, pages, dtype=BF16, seed=0):
    """Each (slots, factor) in turn, caches full of numbers at first."""
    g = torch.Generator().manual_seed(seed)
    bits = [torch.randint(0, 0x70, (pages, Hkv, page, d), generator=g, dtype=torch.uint8) for _ in range(2)]
    exps = [torch.randint(-9, -3, (pages, Hkv), generator=g) for _ in range(2)]
    ref = [b.view(torch.float8_e4m3fn).double() for b in bits]
    caches = [b.cuda().view(torch.float8_e4m3fn) for b in bits]
    scales = [torch.exp2(e.double()).float().cuda() for e in exps]
    for slots, factor in calls:
        gone = left_out(slots, page, pages)
        kept = [-1 if t in gone else s for t, s in enumerate(slots)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        k, v = ((torch.randn(len(slots), Hkv, d, generator=g) * factor).to(dtype) for _ in range(2))
        ea.attn_cache_append_fp8(k.cuda(), v.cuda(), *caches, *scales, torch.tensor(slots, device="cuda"), dev_status=status)
        for x, c, e in zip((k, v), ref, exps):
            ref_append_fp8(x, c, e, kept, page)
        for c, s, rc, re in zip(caches, scales, ref, exps):
            assert torch.equal(torch.exp2(re.double()).float(), s.cpu())
            assert torch.equal(c.double().cpu(), rc)
        bad = bool(gone) or any(s != -1 and not 0 <= s < page * pages for s in slots)
        assert int(status.item()) == int(bad)


# slots of pages of 16 rows, and the tokens that are left out
CASES = [
    ([16, 17, -1, 19], {3}), ([18, 19, -1, -1, -1, 23, 24, -1], {5, 6}), ([-1, 17, -1, 35], set()),
    ([17, -1, -1, -1, 21, 22], {4, 5}), ([24, -1, 26, -1, 28, 40, 41, 56], {2, 4}),
    ([16, 16, 40], {1}), ([18, 17, 18, 40], {1, 2}), ([17, 19, 20, 40], {1, 2}), ([17, 16, 40, 41], {1}),
    ([17, -1, 18, 40], {2}), ([0, 16, 32, 48], set()), ([15, 16, 17, 31], {3}), ([15, -1, 17, 18], set()),
    ([20, -2, 22, 300, 40], {2}), ([16, 17, 33, -1, -1, 40], {5}),
]


@pytest.mark.parametrize("slots,gone", CASES, ids=str)
def test_left_out(slots, gone):
    assert left_out(slots, 16, 8) == gone


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_second_runs_are_left_out_and_reported(dtype, d):
    for slots, _ in CASES:
        append_and_check([(slots, 30.0), (slots, 0.01), (slots, 2000.0 if dtype is BF16 else 100.0)], 2, d, 16, 8, dtype,
                         seed=len(slots))


@gpu
@pytest.mark.parametrize("page", [8, 24, 128, 384])
def test_second_runs_in_long_pages(page):
    """Behind stretches without a slot of every length that is looked for, also longer than
    what a CTA looks at; and just beyond a page's border."""
    for row in sorted({1, 2, 7, page // 2, page - 2}):
        for first in sorted({0, 1, row - 1} - {row}):
            if first >= row:
                continue
            gap = row - first - 1
            slots = [3 * page, page + first] + [-1] * gap + [page + row, page + row + 1 if row + 1 < page else 2 * page]
            append_and_check([(slots, 5.0), ([-1] * 3 + slots, 50.0)], 1, 64, page, 5, seed=row)
        slots = [page - 1] + [-1] * row + [page + row, 3 * page]   # the page before: no second run
        assert left_out(slots, page, 5) == set()
        append_and_check([(slots, 5.0)], 1, 64, page, 5, seed=row)


@gpu
def test_padded_batches():
    """Requests padded to as many tokens each: every run begins behind padding."""
    g = torch.Generator().manual_seed(5)
    for width in (4, 9, 40):
        slots = []
        for b in range(60):
            n = int(torch.randint(0, width + 1, (1,), generator=g))
            r = int(torch.randint(0, 64 - n, (1,), generator=g))
            slots += [b * 64 + r + i for i in range(n)] + [-1] * (width - n)
        assert not left_out(slots, 64, 60)
        append_and_check([(slots, 1.0), (slots, 10.0)], 2, 128, 64, 60, seed=width)
