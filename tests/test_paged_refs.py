"""The paged-cache operators on the CPU: refusals of the C entry points and the
binding, workspace sizes, and the references that the GPU tests use."""
import math
import os

import pytest
import torch

import exact_attention_58_gb300 as ea
from exact_attention_58_gb300 import _build
from paged_ref import check_attention, make_paged, ref_attention, ref_page_table

FAKE = 0x10000   # aligned, never dereferenced: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ea.LIB_PATH):
        _build.build()
    return ea.library()


def paged(lib, **kw):
    a = dict(Q=FAKE, kc=FAKE, vc=FAKE, O=FAKE, LSE=FAKE, cu=FAKE, seq=FAKE, table=FAKE, B=2, H=8,
             Hkv=2, total=2, max_q=1, pages=10, page=16, width=100, d=128, dtype=0, qt=1024, qh=128,
             sp=4096, sh=2048, st=128, scale=0.1, causal=1, window=0, ws=FAKE, wsb=1 << 40, dev=None,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.attn_fwd_paged(*a.values())


@pytest.mark.parametrize("kw,expected", [
    (dict(Q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(O=None), 1),
    (dict(LSE=None), 1), (dict(cu=None), 1), (dict(seq=None), 1), (dict(table=None), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(Hkv=0), 1), (dict(H=7), 1), (dict(total=0), 1),
    (dict(max_q=0), 1), (dict(max_q=-3), 1), (dict(pages=0), 1), (dict(page=0), 1),
    (dict(width=0), 1), (dict(dtype=9), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(d=96), 2), (dict(d=32), 2), (dict(dtype=1), 2), (dict(dtype=3), 2), (dict(page=12), 2),
    (dict(H=258), 2), (dict(width=1 << 27), 2), (dict(pages=1 << 28), 2),
    (dict(total=(1 << 30) + 1), 2), (dict(B=(1 << 30) + 1), 2),
    (dict(B=(1 << 30) - 100, H=2, total=65, max_q=65), 2),   # 2^31 - 200 tiles
    (dict(Q=FAKE + 8), 3), (dict(kc=FAKE + 2), 3), (dict(O=FAKE + 4), 3), (dict(LSE=FAKE + 4), 3),
    (dict(cu=FAKE + 2), 3), (dict(seq=FAKE + 1), 3), (dict(table=FAKE + 2), 3),
    (dict(qt=1020), 3), (dict(qh=0), 3), (dict(sp=-8), 3), (dict(sh=12), 3), (dict(st=1 << 40), 3),
    (dict(ws=None, width=10000), 4), (dict(wsb=100, width=10000), 4),
    (dict(ws=None, max_q=2, total=4, H=128, width=10000), 4),
])
def test_attention_refusals(lib, kw, expected):
    assert paged(lib, **kw) == expected


def append(lib, **kw):
    a = dict(K=FAKE, V=FAKE, kc=FAKE, vc=FAKE, slots=FAKE, T=4, Hkv=2, d=128, dtype=0, ts=256, hs=128,
             pages=10, page=16, sp=4096, sh=2048, st=128, dev=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.attn_cache_append(*a.values())


@pytest.mark.parametrize("kw,expected", [
    (dict(K=None), 1), (dict(V=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(slots=None), 1), (dict(T=0), 1), (dict(Hkv=0), 1), (dict(pages=0), 1), (dict(dtype=7), 1),
    (dict(dtype=1), 2), (dict(dtype=3), 2), (dict(d=80), 2), (dict(page=4), 2),
    (dict(pages=1 << 28), 2),
    (dict(K=FAKE + 8), 3), (dict(vc=FAKE + 8), 3), (dict(slots=FAKE + 4), 3), (dict(ts=250), 3),
    (dict(hs=0), 3), (dict(st=4), 3),
])
def test_append_refusals(lib, kw, expected):
    assert append(lib, **kw) == expected


def table(lib, **kw):
    a = dict(cached=0x1000, new=0x2000, table=0x3000, free=0x4000, num=0x5000, cu=0x6000, seq=0x7000,
             slots=0x8000, taken=0x9000, B=4, width=8, page=16, tokens=64, cap=32, dev=None,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.attn_page_table(*a.values())


@pytest.mark.parametrize("kw,expected", [
    (dict(cached=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(free=None), 1),
    (dict(num=None), 1), (dict(cu=None), 1), (dict(seq=None), 1), (dict(slots=None), 1),
    (dict(taken=None), 1), (dict(B=0), 1), (dict(width=0), 1), (dict(page=0), 1),
    (dict(tokens=0), 1), (dict(cap=0), 1),
    (dict(B=16385), 2), (dict(page=20), 2), (dict(width=1 << 27), 2),
    (dict(cached=0x1002), 3), (dict(slots=0x8004), 3), (dict(taken=0x9001), 3),
    # outputs inside inputs
    (dict(seq=0x1000), 1), (dict(cu=0x1000 - 16), 1), (dict(taken=0x5000), 1),
    (dict(slots=0x4000 - 8), 1), (dict(seq=0x6004), 1), (dict(taken=0x8000), 1), (dict(seq=0x3000 + 4 * 31), 1), (dict(table=0x1008), 1),
])
def test_table_refusals(lib, kw, expected):
    assert table(lib, **kw) == expected


def test_workspace_sizes(lib):
    size = ea.attn_fwd_paged_workspace_size
    assert size(1, 8, 2, 1, 1, 10000, 16, 128) > 0        # one request: its keys are shared out
    assert size(1, 8, 2, 1, 1, 100, 16, 128) == 0         # among a cluster, if they are few
    assert size(1, 8, 2, 200, 200, 10000, 16, 128) > 0 == size(1, 8, 2, 200, 200, 100, 16, 128)
    assert size(4, 16, 16, 4 * 4096, 4096, 32, 128, 128) == 0   # enough tiles without
    # single tokens beside a chunk: the pieces of the single tokens'
    assert size(64, 32, 8, 575, 512, 800, 16, 128) == size(64, 32, 8, 64, 4, 800, 16, 128) > 0
    # ... whose tiles' numbers fit 32 bits: 2^27 rows and more go to one kernel
    assert size(64, 1, 1, (1 << 27) - 1, 1 << 27, 800, 16, 64) > 0 == size(64, 1, 1, 1 << 27, 1 << 27, 800, 16, 64)
    for bad in (dict(B=0), dict(H=7), dict(d=96), dict(max_pages=0)):
        a = dict(B=1, H=8, Hkv=2, total_q=1, max_seqlen_q=1, max_pages=100, page_size=16, d=128)
        a.update(bad)
        assert size(**a) == 0
    # bounded whatever the batch: partial results of at most a wave of CTAs
    for B in (1, 3, 17, 100, 1000):
        for q in (1, 5, 40, 500):
            for d in (64, 128, 256):
                assert size(B, 16, 4, B * q, q, 4096, 16, d) < 256 << 20


def cpu_args():
    x = make_paged([1, 2], [20, 9], 4, 2, 64, 16)
    return x, [x.q, x.k_cache, x.v_cache, x.page_table, x.seq_lens, x.cu]


def test_binding_refuses(lib):
    x, args = cpu_args()
    refused = lambda: pytest.raises(ValueError, match="^(?!.*on a CUDA device)")  # noqa: E731
    with pytest.raises(ValueError, match="on a CUDA device"):   # the last check
        ea.attn_fwd_paged(*args, 2)
    wrong = {0: [x.q[0], x.q.float(), x.q.transpose(1, 2)],
             1: [x.k_cache[0], x.k_cache.half(), x.k_cache[..., :32], x.k_cache[:, :1]],
             2: [x.v_cache[:1], x.v_cache.transpose(1, 2).contiguous().transpose(1, 2)],
             3: [x.page_table.long(), x.page_table[0], x.page_table.t()],
             4: [x.seq_lens.long(), x.seq_lens[:1]],
             5: [x.cu[:2], x.cu.float()]}
    for i, bad in wrong.items():
        for t in bad:
            with refused():
                ea.attn_fwd_paged(*args[:i], t, *args[i + 1:], 2)
    with refused():
        ea.attn_fwd_paged(*args, 2**32 + 1)
    with refused():
        ea.attn_fwd_paged(*args, 2, window=2**32 + 5)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    for bad in [(k, k[:2], slots), (k, k.transpose(0, 1).contiguous().transpose(0, 1), slots),
                (k, k, slots.int()), (k, k, slots[:2]), (k[:, :1], k[:, :1], slots),
                (k, k.half(), slots), (k[0], k[0], slots), (k.float(), k.float(), slots)]:
        with refused():
            ea.attn_cache_append(bad[0], bad[1], x.k_cache, x.v_cache, bad[2])
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    good = [i(1, 2), i(1, 1), x.page_table, i(1, 2, 3), i(3)]
    for at, t in [(0, i(1)), (1, i(1, 1).long()), (2, x.page_table[0]), (3, i(1, 2).reshape(1, 2)),
                  (4, i(3, 3))]:
        with refused():
            ea.attn_page_table(*good[:at], t, *good[at + 1:], 16, 8)
    for tail in [(2**31, 8), (16, 2**31)]:
        with refused():
            ea.attn_page_table(*good, *tail)
    with pytest.raises(ValueError, match="on a CUDA device"):
        ea.attn_page_table(*good, 16, 8)
    with pytest.raises(ValueError, match="on a CUDA device"):
        ea.attn_cache_append(k, k, x.k_cache, x.v_cache, slots)


def test_reference_attention_against_closed_forms():
    """Equal keys give the mean of the values; one key gives its value; a query
    before the first key gives nothing."""
    x = make_paged([1, 3], [7, 2], 4, 2, 64, 8, seed=1)
    x.keys = [torch.zeros_like(k) for k in x.keys]
    O, lse, tol, _ = ref_attention(x, True)
    assert torch.allclose(O[0, 3], x.values[0][:, 1].mean(0), atol=1e-12)
    assert math.isclose(float(lse[0, 0]), math.log(7), abs_tol=1e-12)
    assert bool((O[1] == 0).all()) and bool((lse[:, 1] == -math.inf).all())   # position -1
    assert torch.allclose(O[2, 0], x.values[1][0, 0], atol=1e-12)
    O, _, _, _ = ref_attention(x, True, window=1)
    assert torch.allclose(O[0, 0], x.values[0][6, 0], atol=1e-12)


def test_reference_cache_holds_the_keys():
    x = make_paged([1, 4], [37, 50], 4, 2, 64, 24, seed=3, poison=math.nan)
    for b, L in enumerate([37, 50]):
        ids = x.page_table[b][: -(-L // 24)].long()
        k = x.k_cache[ids].transpose(1, 2).reshape(-1, 2, 64)
        assert torch.equal(k[:L].double(), x.keys[b]) and bool(k[L:].isnan().all())


def test_planted_mistakes_are_seen():
    """An off-by-one in the causal limit, a wrong head, a lost key and a wrong
    normaliser all leave the tolerance."""
    x = make_paged([5, 1], [300, 40], 4, 2, 64, 16, seed=4)
    O, lse, _, _ = ref_attention(x, True)
    check_attention(O, lse, x, True)
    for mistake in ("future", "head", "lost", "sum"):
        y = make_paged([5, 1], [300, 40], 4, 2, 64, 16, seed=4)
        o, z = O.clone(), lse.clone()
        if mistake == "future":
            o, z, _, _ = ref_attention(y, False)
        elif mistake == "head":
            o = O[:, [1, 2, 3, 0]]
        elif mistake == "lost":
            y.keys[0], y.values[0] = y.keys[0][1:], y.values[0][1:]
            o, z, _, _ = ref_attention(y, True)
        else:
            o = O * 1.02
        with pytest.raises(AssertionError):
            check_attention(o, z, x, True)


def test_reference_table():
    cu, seq, slots, taken, t = ref_page_table([3, 16], [2, 1], [[5, -7], [2, -7]], [9, 8, 1], 2, 16, 5)
    assert (cu, seq, taken) == ([0, 2, 3], [5, 17], 1)
    assert slots == [5 * 16 + 3, 5 * 16 + 4, 8 * 16, -1, -1]
    assert t == [[5, -7], [2, 8]]
