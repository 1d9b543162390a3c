"""Paged-cache calls beside the backward's stages on one stream: each kernel may
be resident before the one ahead of it has finished, and none reads what that one
still writes."""
import pytest
import torch

import exact_attention_58_gb300 as ea

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def randn(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(BF16)


def stages(q, k, v, o, do, lse, before_main=()):
    """dQ, dK, dV by the three stages, with calls put in before the main one."""
    B, H, N, d = q.shape
    ws = torch.empty(ea.attn_bwd_workspace_size(B, H, N, d), dtype=torch.uint8, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    torch.cuda.synchronize()
    ea.attn_bwd_preprocess(o, do, lse, ws)
    for call in before_main:
        call()
    ea.attn_bwd_main(q, k, v, do, dk, dv, ws, causal=True)
    ea.attn_bwd_dq_convert(dq, ws)
    torch.cuda.synchronize()
    return dq, dk, dv


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("convert_between", [False, True])
def test_main_stage_behind_a_cache_append(d, convert_between):
    """Contiguous pages are a dense [B, H, N, d]: K and V of the main stage are
    rows that the append right ahead of it (or ahead of another stage) writes,
    the first pages last."""
    B, H, N = 8, 8, 1024
    q, k, v, do = (randn(B, H, N, d, seed=s) for s in range(4))
    o, lse = ea.attn_fwd(q, k, v, causal=True)
    ref = stages(q, k, v, o, do, lse)
    slots = torch.arange(B * N - 1, -1, -1, device="cuda")
    new_k, new_v = (t.transpose(1, 2).reshape(B * N, H, d).flip(0).contiguous() for t in (k, v))
    other = torch.zeros(ea.attn_bwd_workspace_size(1, 1, 128, d), dtype=torch.uint8, device="cuda")
    spare = torch.empty(1, 1, 128, d, dtype=BF16, device="cuda")
    old = randn(B, H, N, d, seed=9)
    for _ in range(5):
        kc, vc = old.clone(), old.clone()
        calls = [lambda: ea.attn_cache_append(new_k, new_v, kc, vc, slots)]
        if convert_between:
            calls.append(lambda: ea.attn_bwd_dq_convert(spare, other))
        got = stages(q, kc, vc, o, do, lse, calls)
        assert torch.equal(kc, k) and torch.equal(vc, v)
        assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])
        assert (got[0].float() - ref[0].float()).abs().max().item() <= 1e-2   # atomic order may differ


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("keys", [40, 700])
def test_main_stage_behind_paged_attention(d, keys):
    """The queries of the main stage are the output of the paged attention right
    ahead of it: one head, one token a request."""
    N, page = 1024, 16
    need = -(-keys // page)
    kc, vc = randn(4 * need, 1, page, d, seed=1), randn(4 * need, 1, page, d, seed=2)
    # four requests' pages, shared by all
    table = torch.arange(4 * need, dtype=torch.int32, device="cuda").view(4, need).repeat(N // 4, 1).contiguous()
    lens = torch.full((N,), keys, dtype=torch.int32, device="cuda")
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    tokens = randn(N, 1, d, seed=3)
    made, _ = ea.attn_fwd_paged(tokens, kc, vc, table, lens, cu, 1, causal=True)
    q = made.view(1, 1, N, d).clone()
    k, v, do = (randn(1, 1, N, d, seed=s) for s in (4, 5, 6))
    o, lse = ea.attn_fwd(q, k, v, causal=True)
    ref = stages(q, k, v, o, do, lse)
    for _ in range(5):
        buf = randn(1, 1, N, d, seed=7)
        got = stages(buf, k, v, o, do, lse,
                     [lambda: ea.attn_fwd_paged(tokens, kc, vc, table, lens, cu, 1, causal=True,
                                                out=buf.view(N, 1, d))])
        assert torch.equal(buf, q)
        assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])
