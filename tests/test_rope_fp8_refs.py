"""Rotary positions and the 8-bit paged cache on the CPU: refusals of the C entry
points and of the binding, frequencies, the references, and planted mistakes."""
import math
import os

import pytest
import torch

import exact_attention_58_gb300 as ea
from exact_attention_58_gb300 import _build
from rope_fp8_ref import check_fp8, fit, make_fp8, ref_append_fp8, ref_rope, rope_tol, round_e4m3

FAKE = 0x10000   # aligned, never dereferenced: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ea.LIB_PATH):
        _build.build()
    return ea.library()


def call(fn, defaults, kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


ROPE = dict(Q=FAKE, K=FAKE, Qo=FAKE, Ko=FAKE, freq=FAKE, pos=FAKE, B=2, H=4, Hk=2, N=10, d=64, r=64, dtype=0,
            qb=2560, qh=640, qt=64, kb=1280, kh=640, kt=64, ob=2560, oh=640, ot=64, pb=1280, ph=640, pt=64,
            pos_b=10, scaling=1.0, inter=0, inv=0, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(Q=None), 1), (dict(Qo=None), 1), (dict(K=None), 1), (dict(Ko=None), 1), (dict(freq=None), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(Hk=-1), 1), (dict(N=0), 1), (dict(r=0), 1), (dict(r=80), 1),
    (dict(dtype=9), 1), (dict(scaling=math.nan), 1), (dict(scaling=math.inf), 1), (dict(pos_b=9), 1), (dict(pos_b=-10), 1),
    (dict(dtype=3), 2), (dict(d=96), 2), (dict(r=24), 2), (dict(N=(1 << 30) + 1), 2), (dict(B=1 << 29), 2),
    (dict(Q=FAKE + 8), 3), (dict(Ko=FAKE + 4), 3), (dict(freq=FAKE + 2), 3), (dict(pos=FAKE + 1), 3),
    (dict(qt=60), 3), (dict(kh=-640), 3), (dict(ot=0), 3), (dict(oh=4), 3), (dict(pb=1 << 40), 3),
])
def test_rope_refusals(lib, kw, expected):
    assert call(lib.attn_rope, ROPE, kw) == expected


APPEND_ROPE = dict(Q=FAKE, K=FAKE, V=FAKE, Qo=FAKE, kc=FAKE, vc=FAKE, slots=FAKE, freq=FAKE, pos=None, cu=FAKE,
                   lens=FAKE, B=2, T=4, H=4, Hkv=2, d=128, r=128, dtype=0, qt=512, qh=128, kt=256, kh=128, ot=512,
                   oh=128, pages=10, page=16, sp=4096, sh=2048, st=128, scaling=1.0, inter=0, dev=None, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(Q=None), 1), (dict(V=None), 1), (dict(Qo=None), 1), (dict(vc=None), 1), (dict(slots=None), 1),
    (dict(freq=None), 1), (dict(cu=None), 1), (dict(lens=None), 1), (dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1),
    (dict(Hkv=0), 1), (dict(pages=0), 1), (dict(page=0), 1), (dict(r=129), 1), (dict(scaling=math.nan), 1), (dict(dtype=7), 1),
    (dict(dtype=1), 2), (dict(dtype=3), 2), (dict(d=80), 2), (dict(r=8), 2), (dict(page=12), 2), (dict(pages=1 << 28), 2),
    (dict(T=(1 << 30) + 1), 2),
    (dict(K=FAKE + 8), 3), (dict(slots=FAKE + 4), 3), (dict(qt=500), 3), (dict(st=0), 3), (dict(oh=0), 3), (dict(lens=FAKE + 2), 3),
])
def test_append_rope_refusals(lib, kw, expected):
    assert call(lib.attn_cache_append_rope, APPEND_ROPE, kw) == expected


APPEND8 = dict(K=FAKE, V=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, slots=FAKE, T=4, Hkv=2, d=128, dtype=0, ts=256,
               hs=128, pages=10, page=16, sp=4096, sh=2048, st=128, dev=None, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(K=None), 1), (dict(vc=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(slots=None), 1),
    (dict(T=0), 1), (dict(Hkv=0), 1), (dict(pages=0), 1), (dict(dtype=7), 1),
    (dict(dtype=1), 2), (dict(dtype=3), 2), (dict(d=80), 2), (dict(page=4), 2), (dict(pages=1 << 28), 2), (dict(T=1 << 30), 2),
    (dict(K=FAKE + 8), 3), (dict(vc=FAKE + 8), 3), (dict(ks=FAKE + 2), 3), (dict(slots=FAKE + 4), 3),
    (dict(ts=250), 3), (dict(sp=4104), 3), (dict(st=8), 3),
])
def test_append_fp8_refusals(lib, kw, expected):
    assert call(lib.attn_cache_append_fp8, APPEND8, kw) == expected


PAGED8 = dict(Q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, O=FAKE, LSE=FAKE, cu=FAKE, seq=FAKE, table=FAKE, B=2, H=8,
              Hkv=2, total=2, max_q=1, pages=10, page=16, width=100, d=128, dtype=0, qt=1024, qh=128, sp=4096,
              sh=2048, st=128, scale=0.1, causal=1, window=0, ws=FAKE, wsb=1 << 40, dev=None, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(Q=None), 1), (dict(kc=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(O=None), 1),
    (dict(table=None), 1), (dict(B=0), 1), (dict(H=7), 1), (dict(total=0), 1), (dict(scale=0.0), 1),
    (dict(scale=math.nan), 1), (dict(dtype=9), 1),
    (dict(d=96), 2), (dict(dtype=1), 2), (dict(dtype=3), 2), (dict(page=12), 2), (dict(H=258), 2), (dict(width=1 << 27), 2),
    (dict(Q=FAKE + 8), 3), (dict(vs=FAKE + 1), 3), (dict(LSE=FAKE + 4), 3), (dict(sp=4104), 3), (dict(st=8), 3),
    (dict(qt=1020), 3), (dict(ws=None, width=10000), 4), (dict(wsb=100, width=10000), 4),
])
def test_attention_refusals(lib, kw, expected):
    assert call(lib.attn_fwd_paged_fp8, PAGED8, kw) == expected


def refused():
    return pytest.raises(ValueError, match="^(?!.*on a CUDA device)")


def last():
    return pytest.raises(ValueError, match="on a CUDA device")


def test_binding_refuses(lib):
    x = make_fp8([1, 2], [20, 9], 4, 2, 64, 16)
    args = [x.q, x.k_cache, x.v_cache, x.k_scale, x.v_scale, x.page_table, x.seq_lens, x.cu]
    with last():
        ea.attn_fwd_paged_fp8(*args, 2)
    wrong = {0: [x.q[0], x.q.float().transpose(1, 2)], 1: [x.k_cache[0], x.k_cache.float(), x.k_cache[:, :1]],
             2: [x.v_cache[:1]], 3: [x.k_scale.double(), x.k_scale[:, :1], x.k_scale[:-1], None],
             4: [x.v_scale.t()], 5: [x.page_table.long()], 6: [x.seq_lens[:1]], 7: [x.cu.float()]}
    for i, bad in wrong.items():
        for t in bad:
            with refused():
                ea.attn_fwd_paged_fp8(*args[:i], t, *args[i + 1:], 2)
    with refused():   # a 16-bit cache
        ea.attn_fwd_paged_fp8(x.q, x.k_cache.bfloat16(), x.v_cache.bfloat16(), *args[3:], 2)
    k, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    good = [k, k, x.k_cache, x.v_cache, x.k_scale, x.v_scale, slots]
    with last():
        ea.attn_cache_append_fp8(*good)
    for i, t in [(0, k[:, :1]), (1, k.half()), (2, x.k_cache.half()), (4, x.k_scale.half()), (5, x.v_scale[:1]),
                 (6, slots.int())]:
        with refused():
            ea.attn_cache_append_fp8(*good[:i], t, *good[i + 1:])


def test_rope_binding_refuses(lib):
    bf = torch.bfloat16
    q, k, f = torch.zeros(2, 4, 10, 64, dtype=bf), torch.zeros(2, 2, 10, 64, dtype=bf), torch.ones(32)
    with last():
        ea.attn_rope(q, k, f)
    with refused():   # an output for keys that are not there
        ea.attn_rope(q, None, f, k_out=k)
    with last():
        ea.attn_rope(q, None, f, torch.zeros(2, 10, dtype=torch.int32))
    i32 = torch.int32
    for bad in [(q[0], k, f), (q, k[:1], f), (q, k.half(), f), (q, k, f.double()), (q, k, f[None]),
                (q, k, f, torch.zeros(9, dtype=i32)), (q, k, f, torch.zeros(10)), (q, k, f, torch.zeros(2, 9, dtype=i32)),
                (q.transpose(2, 3), k, f), (q[:, 0], q[:, 0], f), (q, k[:, :0], f)]:
        with refused():
            ea.attn_rope(*bad)
    with refused():
        ea.attn_rope(q, k, f, q_out=q[:1])
    t, c = torch.zeros(5, 2, 64, dtype=bf), torch.zeros(3, 2, 16, 64, dtype=bf)
    s, n = torch.zeros(5, dtype=torch.int64), torch.zeros(5, dtype=i32)
    with last():
        ea.attn_cache_append_rope(t, t, t, c, c, s, f, n)
    with last():
        ea.attn_cache_append_rope(t, t, t, c, c, s, f, cu_seqlens_q=n[:3], seq_lens=n[:2])
    for a, kw in [((t[:4], t, t, c, c, s, f, n), {}), ((t, t, t, c, c, s, f), {}),
                  ((t, t, t, c, c, s, f), dict(seq_lens=n[:2])), ((t, t, t, c, c, s, f), dict(cu_seqlens_q=n, seq_lens=n)),
                  ((t, t, t, c.half(), c, s, f, n), {}), ((t, t, t[:, :1], c, c, s, f, n), {})]:
        with refused():
            ea.attn_cache_append_rope(*a, **kw)


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
def test_frequencies():
    f, s = ea.attn_rope_frequencies(128)
    assert s == 1.0 and f.dtype is torch.float32
    assert torch.allclose(f.double(), 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64), rtol=2.0**-23)
    g, s = ea.attn_rope_frequencies(128, factor=4.0)
    assert s == 1.0 and torch.equal(g, f / 4)
    g, s = ea.attn_rope_frequencies(128, factor=4.0, method="base")
    assert s == 1.0 and g[0] == 1 and abs(float(g[-1] * 4 / f[-1]) - 1) < 1e-6
    g, s = ea.attn_rope_frequencies(128, factor=4.0, method="parts", original_len=4096)
    assert abs(s - (0.1 * math.log(4) + 1)) < 1e-12
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 40], f[turns > 40]) and torch.equal(g[turns < 0.8], f[turns < 0.8] / 4)
    assert bool((g <= f).all()) and bool((g >= f / 4 * (1 - 1e-6)).all()) and bool((g[1:] < g[:-1]).all())
    for kw in (dict(factor=0.5), dict(method="other"), dict(base=1.0), dict(method="parts"),
               dict(method="parts", original_len=100, fast=1.0, slow=2.0), dict(factor=math.nan)):
        with pytest.raises(ValueError):
            ea.attn_rope_frequencies(64, **kw)
    for r in (0, 3, -2):
        with pytest.raises(ValueError):
            ea.attn_rope_frequencies(r)


@pytest.mark.parametrize("n", [1, 40, 300, 4096, 131072, 10**7])
@pytest.mark.parametrize("r", [16, 64, 128])
def test_frequencies_by_parts_at_any_length(r, n):
    """Kept from `fast` turns on, divided up to `slow`, mixed in between, also where
    all pairs, or none, lie to one side."""
    f, _ = ea.attn_rope_frequencies(r)
    g, _ = ea.attn_rope_frequencies(r, factor=4.0, method="parts", original_len=n)
    turns = n * f.double() / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32])
    # (a division in 64 bits, rounded, is the exact quotient by a power of two of the rounded)
    assert torch.equal(g[turns <= 1], f[turns <= 1] / 4)
    # strictly between away from the whole indices that the two ends are rounded to
    step = 10000.0 ** (2 / r)
    inside = (turns > 1 * step) & (turns < 32 / step)
    assert bool((g[inside] < f[inside]).all()) and bool((g[inside] > f[inside] / 4).all())


# ---------------------------------------------------------------------------
# references
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
def test_ref_rope(interleaved):
    g = torch.Generator().manual_seed(0)
    f = torch.tensor([1.0, 0.1, 0.01, 0.001])
    x, y = torch.randn(2, 10, generator=g, dtype=torch.float64)
    at = lambda v, p, **kw: ref_rope(v, torch.tensor(p), f, interleaved, **kw)  # noqa: E731
    assert torch.allclose(at(x, 0), x)
    assert torch.equal(at(x, 9)[8:], x[8:])                       # the rest of the row
    dot = lambda a, b: float(at(x, a)[:8] @ at(y, b)[:8])  # noqa: E731
    assert abs(dot(1000, 990) - dot(10, 0)) < 1e-9                # only the distance counts
    assert torch.allclose(at(at(x, 7), 7, inverse=True), x)
    assert abs(float(at(x, 5, scaling=1.5) @ y - x @ at(y, 5, scaling=1.5, inverse=True))) < 1e-12   # the transpose
    one = torch.zeros(10, dtype=torch.float64)
    one[2] = 1.0
    z = at(one, 30)
    b, w = (3, 3.0) if interleaved else (6, 0.3)   # the pair's other element; 30 times its frequency
    assert abs(float(z[2]) - math.cos(w)) < 1e-7 and abs(float(z[b]) - math.sin(w)) < 1e-7
    # differences of the map are the gradient's
    tol = rope_tol(x, at(x, 5), torch.tensor(5), f, interleaved, 1.0, torch.bfloat16)
    wrong = at(x, 6)
    assert bool(((wrong - at(x, 5)).abs() > tol)[:8].any()) and bool((tol[8:] == 0).all())


def test_ref_rounding():
    for x, y in [(0.0, 0.0), (448.0, 448.0), (460.0, 448.0), (-1e9, -448.0), (17.0, 16.0), (19.0, 20.0), (2.0**-10, 0.0),
                 (1.5 * 2.0**-9, 2.0**-8), (2.0**-6, 2.0**-6), (-2.0**-9, -2.0**-9), (math.inf, 448.0), (-math.inf, -448.0)]:
        assert float(round_e4m3(torch.tensor(x, dtype=torch.float64))) == y
    assert math.isnan(float(round_e4m3(torch.tensor(math.nan, dtype=torch.float64))))
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(round_e4m3(every).nan_to_num(7.0), every.nan_to_num(7.0))
    g = torch.Generator().manual_seed(1)
    x = torch.randn(20000, generator=g) * 40
    assert torch.equal(round_e4m3(x.double()), x.clamp(-448, 448).to(torch.float8_e4m3fn).double())
    assert [fit(v) for v in (0.0, 448.0, 448.5, 3.5, 3.51, 1e30, math.inf)] == [-48, 0, 1, -7, -6, 48, 48]


def test_ref_append_grows_and_starts_anew():
    cache, exps = torch.zeros(2, 1, 8, 64, dtype=torch.float64), torch.zeros(2, 1, dtype=torch.int64)
    x = torch.ones(3, 1, 64)
    x[1] *= 100.0
    ref_append_fp8(x[:1], cache, exps, [8], 8)
    assert int(exps[1, 0]) == -8 and float(cache[1, 0, 0, 0]) == 256.0
    ref_append_fp8(x[1:], cache, exps, [9, 10], 8)
    assert int(exps[1, 0]) == -2 and cache[1, 0, :4, 0].tolist() == [4.0, 384.0, 4.0, 0.0]   # 100 = 25 / 2^-2 -> 24 x 16
    ref_append_fp8(x[:1], cache, exps, [8], 8)
    assert int(exps[1, 0]) == -8 and cache[1, 0, :2, 0].tolist() == [256.0, 384.0]
    ref_append_fp8(x[:1], cache, exps, [-1], 8)
    assert exps[:, 0].tolist() == [0, -8]


def plain_attention(x, causal):
    """O, LSE rounded to the storage type, from the references' own formula."""
    from paged_ref import ref_attention
    O, L, _, _ = ref_attention(x, causal)
    return O.to(x.q.dtype), L


@pytest.mark.parametrize("mistake", [None, "k scale", "v scale", "last key", "neighbour's scale"])
def test_planted_mistakes(mistake):
    x = make_fp8([3, 1], [50, 33], 4, 2, 64, 16, spread=1, seed=3)
    y = make_fp8([3, 1], [50, 33], 4, 2, 64, 16, spread=1, seed=3)
    if mistake == "k scale":
        y.keys[0][16:32] *= 2
    elif mistake == "v scale":
        y.values[0][16:32] *= 2
    elif mistake == "last key":
        y.keys[0], y.values[0] = y.keys[0][:-1], y.values[0][:-1]
    elif mistake == "neighbour's scale":
        y.values[0][48:] *= 2
    o, lse = plain_attention(y, False)
    if mistake is None:
        check_fp8(o, lse, x, False)
    else:
        with pytest.raises(AssertionError):
            check_fp8(o, lse, x, False)
