"""np_paged_prefill: one workspace, calls of different batches in a row: a call sees its own plan, not
what an earlier one left (the join begins to read it while the attention runs)."""
import random

import pytest
import torch

from prompt_helpers import chunk_inputs, chunk_reference, chunk_tolerance

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64), (F32, 256)])
def test_batches_in_turn_on_one_workspace(nplib, dtype, d):
    rnd = random.Random(d)
    batches = [[(1, 9000)], [(40, 5000), (3, 3)], [(300, 300)] * 5, [(1, rnd.randint(1, 3000)) for _ in range(50)],
               [(7, 4000), (200, 900)]]
    inps = [chunk_inputs(dtype, d, 2, 2, 16, rows, seed=i) for i, rows in enumerate(batches)]
    ws, scale = nplib.prefill_workspace(d), d ** -0.5
    want = []
    for inp, rows in zip(inps, batches):  # each alone, on a workspace of its own
        out, own = torch.empty_like(inp["q"]), nplib.prefill_workspace(d).zero_()
        nplib.np_paged_prefill(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["block_tables"],
                               inp["context_lens"], inp["query_starts"], scale, own)
        torch.cuda.synchronize()
        ref, bound = chunk_reference(inp, rows, scale)
        tol = chunk_tolerance(ref, bound, dtype, d, max(c for _, c in rows))
        assert ((out.double() - ref).abs() <= tol).all()
        want.append(out)
    order = [rnd.randrange(len(batches)) for _ in range(120)]
    outs = [torch.full_like(want[i], 77.0) for i in order]
    torch.cuda.synchronize()
    for i, out in zip(order, outs):  # back to back, nothing between them
        inp = inps[i]
        nplib.np_paged_prefill(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["block_tables"],
                               inp["context_lens"], inp["query_starts"], scale, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want[i]) for i, out in zip(order, outs))
