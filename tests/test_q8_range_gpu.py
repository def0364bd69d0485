"""The 8-bit reads where blocks' scales lie far apart, against the formula in 64 bits."""
import math

import pytest
import torch

import q8_helpers as h
from prompt_helpers import chunk_reference, chunk_tolerance

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
FORMS = pytest.mark.parametrize("form", [E4M3, INT8], ids=["e4m3", "int8"])
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


def _set(inp, block, *, k=None, v=None, ke=None, ve=None, row=0):
    """Codes (one value for all) and exponents of the row's `block` (an index or a slice)."""
    ids = inp["block_tables"][row][block].long().reshape(-1)
    for name, x in (("k_pool", k), ("v_pool", v)):
        if x is not None:
            pool = inp[name]
            code = torch.tensor(x, dtype=torch.float32).to(pool.dtype).view(torch.uint8)
            pool.view(torch.uint8)[ids] = code.to(pool.device)
    for name, e in (("k_scale", ke), ("v_scale", ve)):
        if e is not None:
            inp[name][ids] = 2.0 ** e


def _decode(npg, inp, scale):
    out = torch.full_like(inp["q"], 7.0)
    npg.np_paged_decode_q8(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["k_scale"], inp["v_scale"],
                           inp["block_tables"], inp["context_lens"], scale,
                           npg.decode_q8_workspace(inp["q"].shape[-1]))
    return out.double()


def _prefill(npg, inp, scale):
    out = torch.full_like(inp["q"], 7.0)
    npg.np_paged_prefill_q8(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["k_scale"], inp["v_scale"],
                            inp["block_tables"], inp["context_lens"], inp["query_starts"], scale,
                            npg.prefill_workspace(inp["q"].shape[-1]))
    return out.double()


def _zero_v_beside_large_v(dtype, form, d, bs, n, c, top, low, where, gap):
    """A row of n tokens over c positions.  All blocks' V is zero under 2^low but that of block
    `where`, under 2^top, whose scores are `gap` higher than the others' in log2 units."""
    inp = h.read_inputs(dtype, form, d, 1, 2, bs, [(n, c)], seed=c)
    inp["q"].fill_(1.0)
    every = slice(0, -(-c // bs))
    v = inp["v_pool"][inp["block_tables"][0][where].long()].clone()
    _set(inp, every, k=0.0, v=0.0, ke=0, ve=low)
    _set(inp, where, k=1.0, ve=top)
    inp["v_pool"][inp["block_tables"][0][where].long()] = v
    return inp, gap * math.log(2.0) / d


# the zero positions' share of the sum is 0.1 to 0.9 of it
SPREADS = [(60, -60, 1016, 0, 6.5), (60, -60, 1016, 60, 6.5), (60, -60, 20000, 700, 9.0),
           (60, -60, 20000, 0, 12.5), (60, -60, 20000, 1200, 12.5), (50, -55, 20000, 0, 9.0),
           (60, -30, 3000, 2, 7.0), (-60, 60, 1016, 3, 5.5), (-20, -21, 300, 3, 3.0), (60, 20, 3000, 9, 7.0)]


@FORMS
@TYPES
@pytest.mark.parametrize("top,low,c,where,gap", SPREADS)
@pytest.mark.parametrize("d", [64, 128])
def test_decode_counts_positions_whose_v_is_far_smaller(nplib, dtype, form, d, top, low, c, where, gap):
    inp, scale = _zero_v_beside_large_v(dtype, form, d, 16, 1, c, top, low, where, gap)
    out = _decode(nplib, inp, scale)
    ref, bound = chunk_reference(h.as_values(inp), [(1, c)], scale)
    tol = h.decode_tolerance(ref, bound, dtype, d, c, 2.0 ** top * h.QMAX[form])
    worst = ((out - ref).abs() / tol).nan_to_num(nan=9e9).max().item()
    assert worst <= 1, worst
