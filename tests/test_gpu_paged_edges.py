"""Paged-cache calls at the ends of their ranges on the GPU: bad lengths inside
guard bands, and token buffers that take a second turn of the page table's grid."""
import pytest
import torch

import exact_attention_58_gb300 as ea
from paged_ref import check_attention, make_paged, ref_page_table
from test_gpu_paged import make_table, run_table

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
BAND = 4096


@pytest.mark.parametrize("cu,seq,good", [
    ([0, 3, 2], [50, 60], None), ([0, 1, 99], [50, 60], None), ([-4, 1, 2], [50, 60], 1),
    ([0, 20, 31], [-1, 60], 1), ([0, 20, 31], [50, 1 << 30], 0), ([0, 30, 31], [50, 60], 1),
    ([0, 20, 31], [2**31 - 1, 60], 1), ([0, 2**31 - 1, 31], [50, 60], None),
    ([0, 20, -2**31], [50, 60], 0),
], ids=str)
@pytest.mark.parametrize("max_q", [1, 3, 20])
@pytest.mark.parametrize("width", [0, 8000], ids=["short table", "wide table"])
def test_bad_lengths_write_inside_the_outputs_and_are_reported(cu, seq, good, max_q, width):
    """Whatever the offsets and lengths say, nothing is written outside O and LSE,
    the call is reported, and a request whose own lengths are right gets its
    result."""
    x = make_paged([20, 11], [50, 60], 4, 2, 64, 16, seed=12)
    n = x.q.numel()
    buf = torch.full((n + 2 * BAND,), 3.0, dtype=BF16, device="cuda")
    lbuf = torch.full((4 * 31 + 2 * BAND,), 3.0, device="cuda")
    out, lse = buf[BAND:BAND + n].view(x.q.shape), lbuf[BAND:-BAND].view(4, -1)
    table = torch.nn.functional.pad(x.page_table, (0, width), value=-1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ea.attn_fwd_paged(x.q.cuda(), x.k_cache.cuda(), x.v_cache.cuda(), table.cuda(), i32(seq), i32(cu),
                      max_q, causal=True, out=out, lse=lse, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 1
    for b in (buf, lbuf):
        assert bool((b[:BAND] == 3).all()) and bool((b[-BAND:] == 3).all())
    if good is None or cu[good + 1] - cu[good] > max_q:
        return
    # the good request alone: its rows, its lengths
    a, e = cu[good], cu[good + 1]
    y = make_paged([20, 11], [50, 60], 4, 2, 64, 16, seed=12)
    y.q, y.keys, y.values = x.q[a:e], [x.keys[good]], [x.values[good]]
    y.cu = torch.tensor([0, e - a], dtype=torch.int32)
    check_attention(out[a:e], lse[:, a:e], y, True)


@pytest.mark.parametrize("new,cached,pad", [
    ([200000, 100000, 50000], [5, 160, 33], 0), ([311296, 1, 40], [0, 15, 16], 300000)], ids=str)
def test_page_table_of_many_tokens(new, cached, pad):
    """More tokens than the grid has threads (608 x 512): each takes several."""
    page = 16
    table, free, _ = make_table(cached, new, page, seed=5)
    T = sum(new) + pad
    got, status = run_table(cached, new, table, free, len(free), page, T)
    assert got == ref_page_table(cached, new, table, free, len(free), page, T)
    assert status == 0
