"""np_paged_prefill: what the roles of a block hand one another.

Scores, weights and sums share tensor memory and its products run asynchronously, so a missing wait
between two of them shows as bits that change, or as values that are off where the timing is unlucky:
the same call many times, alone and with another call beside it, always the same bits; its first
result against 64 bits."""
import random

import pytest
import torch

from prompt_helpers import chunk_inputs, chunk_reference, chunk_tolerance

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rows(seed):
    """Units of one tile with one warp of rows or with all, short ones, and units of two tiles of
    which the first ends tiles before the second."""
    rnd = random.Random(seed)
    rows = [(1, rnd.randint(1, 1500)) for _ in range(20)] + [(n, n + rnd.randint(0, 900)) for n in
                                                            (3, 17, 30, 33, 64, 65, 127, 130, 400)]
    rnd.shuffle(rows)
    return rows


@pytest.mark.parametrize("dtype,d,hk,g,bs", [(BF, 128, 4, 1, 16), (BF, 128, 2, 5, 8), (BF, 128, 2, 8, 5),
                                             (BF, 64, 3, 4, 32), (BF, 16, 2, 4, 16), (BF, 256, 2, 4, 16),
                                             (F32, 128, 2, 4, 16), (F32, 32, 2, 1, 16)])
def test_the_same_bits_a_hundred_times(nplib, dtype, d, hk, g, bs):
    rows, scale = _rows(d + g), d ** -0.5
    inp = chunk_inputs(dtype, d, hk, g, bs, rows, seed=d + g)
    ws, ws2 = (nplib.prefill_workspace(d).fill_(255) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(out, w, stream=None):
        nplib.np_paged_prefill(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["block_tables"],
                               inp["context_lens"], inp["query_starts"], scale, w, err_word=err,
                               stream=stream)
        return out

    want = call(torch.full_like(inp["q"], 77.0), ws)
    torch.cuda.synchronize()
    ref, bound = chunk_reference(inp, rows, scale)
    tol = chunk_tolerance(ref, bound, dtype, d, max(c for _, c in rows))
    assert ((want.double() - ref).abs() <= tol).all()
    outs = [torch.full_like(want, 77.0) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    differs = torch.zeros(1, dtype=torch.bool, device="cuda")
    torch.cuda.synchronize()
    for _ in range(50):
        for o, w, s in zip(outs, (ws, ws2), streams):
            call(o, w, s)
        torch.cuda.synchronize()
        for o in outs:
            differs |= (o.view(torch.int16) != want.view(torch.int16)).any()
            o.fill_(77.0)
        torch.cuda.synchronize()
    assert not bool(differs) and int(err) == 0
