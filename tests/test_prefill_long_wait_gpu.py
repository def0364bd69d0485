"""np_paged_prefill: the warps of a block's second q tile have nothing to do in units of one tile, and may
not take a long run of these for a hang.  (A wait that nothing ends gives up after about a second.)"""
import pytest
import torch

from prompt_helpers import chunk_reference, chunk_tolerance

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_a_second_of_one_token_rows_before_a_chunk(nplib):
    d, hk, g, bs, blocks, last = 128, 8, 1, 1024, 8, (300, 300)
    copies = 160
    each = copies * blocks * bs  # the rows' histories go over the same few blocks again and again
    gen = torch.Generator().manual_seed(1)
    kp, vp = (torch.randn(blocks, bs, hk, d, generator=gen).to(BF).cuda() for _ in range(2))
    once = torch.arange(blocks, dtype=torch.int32, device="cuda")
    ws = nplib.prefill_workspace(d)
    q_one = torch.randn(1, hk * g, d, generator=gen).to(BF).cuda()
    q_last = torch.randn(last[0], hk * g, d, generator=gen).to(BF).cuda()

    def call(rows):
        """`rows` one-token rows, then the chunk: (out, milliseconds, flags)."""
        tables = once.repeat(copies).expand(rows + 1, -1).contiguous()
        lens = torch.full((rows + 1,), each, dtype=torch.int32, device="cuda")
        lens[rows] = last[1]
        starts = torch.arange(rows + 2, dtype=torch.int32, device="cuda")
        starts[rows + 1] = rows + last[0]
        q = torch.cat([q_one.expand(rows, -1, -1), q_last])
        out, err = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        nplib.np_paged_prefill(out, q, kp, vp, tables, lens, starts, d ** -0.5, ws, err_word=err)
        b.record()
        torch.cuda.synchronize()
        return out, a.elapsed_time(b), int(err)

    call(40)
    _, ms, err = call(400)
    assert err == 0
    rows = min(4000, int(400 * 1500 / ms) + 1)
    out, ms, err = call(rows)
    assert ms > 1200  # longer than a wait's limit, 2e9 cycles of at most 2.07 GHz: else the case shows nothing
    assert err == 0
    # softmax over copies of a history is softmax over one
    inp = dict(q=torch.cat([q_one, q_last]), k_pool=kp, v_pool=vp,
               block_tables=once.expand(2, -1), query_starts=torch.tensor([0, 1, 1 + last[0]]))
    ref, bound = chunk_reference(inp, [(1, blocks * bs), last], d ** -0.5)
    tol = chunk_tolerance(ref, bound, BF, d, each)
    assert ((out[rows:].double() - ref[1:]).abs() <= tol[1:]).all()
    assert ((out[:rows].double() - ref[:1]).abs() <= tol[:1]).all()
