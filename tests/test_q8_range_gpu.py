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


def _within(inp, rows, scale, out, dtype, tokens=None):
    """Every output as near to the formula as the positions that its own token sees ask for: nothing is
    allowed for other positions' scales.

    What fp16 weights add to prompt_helpers.chunk_tolerance: a weight (softmax times V's scale) is off by
    at most 2^-25 at fp16's small end, where the largest of the row, or 2^-4 of it (a tile's scales are
    one factor where they lie no further apart), is 2^6 or more: 2^-27 of the largest weight times the
    largest code, for each of the positions.  fp32, rows of few tokens: q and the weights in two parts,
    2^-22 each."""
    form, d, bs, longest = inp["v_pool"].dtype, out.shape[-1], inp["k_pool"].shape[1], max(c for _, c in rows)
    values = h.as_values(inp)
    ref, bound = chunk_reference(values, rows, scale)
    tol = chunk_tolerance(ref, bound, dtype, d, longest)
    if dtype is F32:
        tol = tol + 1.1 * (2 * 2.0 ** -22 * bound[1] + 2.0 ** -22) * bound[0]
    g, at = out.shape[1] // inp["k_pool"].shape[2], 0
    for r, (n, c) in enumerate(rows):
        t = torch.arange(c, device="cuda")
        ids = inp["block_tables"][r].long()[t // bs]
        keys, e = values["k_pool"][ids, t % bs], inp["v_scale"][ids].double()  # [c, heads, ..]
        z = torch.einsum("nhgd,chd->nhgc", inp["q"][at:at + n].double().unflatten(1, (-1, g)), keys) * scale
        z.masked_fill_(t > c - n + torch.arange(n, device="cuda")[:, None, None, None], -math.inf)
        largest = (torch.softmax(z, -1) * e.T[:, None]).amax(-1).flatten(1, 2)
        tol[at:at + n] += longest * 2.0 ** -27 * h.QMAX[form] * largest[..., None]
        at += n
    off = ((out - ref).abs() / tol)[:tokens].nan_to_num(nan=9e9)
    assert off.max().item() <= 1, (off.max().item(), int(off.amax(-1).amax(-1).argmax()))


FAR = [3, 4, 5, 8, 15, 16, 20, 24, 25, 30, 40, 68, 100]


@FORMS
@pytest.mark.parametrize("dtype,d,bs", [(BF, 128, 16), (BF, 64, 8), (BF, 256, 64), (BF, 256, 16), (BF, 128, 5),
                                         (F32, 128, 16)])
@pytest.mark.parametrize("e", FAR)
def test_positions_not_yet_seen_change_nothing(nplib, dtype, d, bs, form, e):
    """A prompt whose later tokens' V (then K) has a far larger scale than its first ones'."""
    n = 192
    for name in ("v_scale", "k_scale"):
        # (scores below 2^30 where the large keys are seen)
        scale = 0.05 if name == "v_scale" else 0.05 * 2.0 ** -max(0, e - 20)
        inp = h.read_inputs(dtype, form, d, 2, 2, bs, [(n, n)], seed=e, spread=0)
        b = 64 // bs + 1  # (the first of these blocks begins at 64 at least)
        _set(inp, slice(b, -(-n // bs)), **{"ve" if name == "v_scale" else "ke": min(60, e - 8)})
        if e > 68:
            _set(inp, slice(0, b), **{"ve" if name == "v_scale" else "ke": 60 - e})
        out = _prefill(nplib, inp, scale)
        assert out.isfinite().all()
        _within(inp, [(n, n)], scale, out, dtype, b * bs if name == "k_scale" else n)


@FORMS
@TYPES
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 40, 200])
@pytest.mark.parametrize("e", [10, 30, 60])
def test_large_values_without_weight_change_nothing(nplib, dtype, d, form, n, e):
    """Blocks of a far larger V whose scores leave them no weight, first and in the middle of a history."""
    rows = [(n, 1000)]
    inp = h.read_inputs(dtype, form, d, 2, 2, 16, rows, seed=n, spread=0)
    inp["q"].fill_(1.0)
    for b in (0, 30):
        _set(inp, b, k=-2.0, ke=8, ve=e)
    out = _prefill(nplib, inp, 0.02)  # the blocks' scores: -655 and below
    ref, bound = chunk_reference(h.as_values(inp), rows, 0.02)
    # (their products' sizes do not count: the others' scores are of ordinary ones)
    keep = [j for j in range(63) if j not in (0, 30)]
    few = dict(inp, block_tables=inp["block_tables"][:, keep].contiguous())
    # the same row without the blocks: the same formula but for weights of e^-655
    _within(few, [(n, 1000 - 32)], 0.02, out, dtype)
    assert (ref - out).isfinite().all() and bound[0].isfinite().all()


@FORMS
@TYPES
@pytest.mark.parametrize("n", [1, 20, 300])
@pytest.mark.parametrize("top,low,c,where,gap", SPREADS)
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 16), (256, 16), (128, 5)])
def test_chunks_count_positions_whose_v_is_far_smaller(nplib, dtype, form, d, bs, n, top, low, c, where, gap):
    if c < n:
        n = c
    inp, scale = _zero_v_beside_large_v(dtype, form, d, bs, n, c, top, low, where, gap)
    out = _prefill(nplib, inp, scale)
    _within(inp, [(n, c)], scale, out, dtype)


@pytest.mark.parametrize("dtype,d,g", [(BF, 64, 1), (BF, 64, 16), (BF, 128, 3), (BF, 128, 8), (BF, 256, 5), (F32, 128, 4)])
@pytest.mark.parametrize("bs,scale", [(8, -0.06), (24, 0.06), (64, -0.06), (256, 0.06)])
def test_far_scales_in_every_shape(nplib, dtype, d, g, bs, scale):
    """Blocks of K up to 2^6 and of V up to 2^46 apart, in ragged chunks, short rows among them."""
    rows = [(5, 5), (1, 300), (130, 700), (64, 64), (33, 1000), (2, 2), (257, 257), (90, 2100)]
    form = E4M3 if bs in (8, 64) else INT8
    inp = h.read_inputs(dtype, form, d, 2, g, bs, rows, seed=bs + g, spread=3)
    gen = torch.Generator().manual_seed(bs)
    inp["v_scale"] *= torch.ldexp(torch.ones(inp["v_scale"].shape),
                                  torch.randint(-20, 21, inp["v_scale"].shape, generator=gen)).cuda()
    out = _prefill(nplib, inp, scale)
    _within(inp, rows, scale, out, dtype)
