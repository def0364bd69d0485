"""np_paged_decode_q8 against the formula in 64 bits."""
import pytest
import torch

import q8_helpers as h
from prompt_helpers import chunk_reference

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _read(npg, inp, rows, scale, ql, stream=None):
    q = inp["q"]
    if ql > 1:
        q = q.view(len(rows), ql, *q.shape[1:])
    out = torch.full_like(q, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((npg.np_paged_decode_q8_workspace_bytes(q.shape[-1]),), 0xff, dtype=torch.uint8, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    npg.np_paged_decode_q8(out, q, inp["k_pool"], inp["v_pool"], inp["k_scale"], inp["v_scale"],
                           inp["block_tables"], inp["context_lens"], scale, ws, err_word=err,
                           stream=stream)
    torch.cuda.synchronize()
    return out.view(inp["q"].shape), int(err)


def _compare(npg, dtype, form, d, hk, g, bs, lens, ql=1, seed=0, scale=None, spread=2):
    rows = [(ql, c) for c in lens]
    inp = h.read_inputs(dtype, form, d, hk, g, bs, rows, seed=seed, spread=spread)
    scale = d ** -0.5 / 2 if scale is None else scale
    out, err = _read(npg, inp, rows, scale, ql)
    assert err == 0
    # a chunk of more tokens than positions: the reference's rows count from the end too
    ref, bound = chunk_reference(h.as_values(inp), rows, scale)
    used = inp["v_scale"][inp["block_tables"][inp["block_tables"] >= 0].long()]
    vtop = float(used.max()) * h.QMAX[form] if used.numel() else 0.0
    tol = h.decode_tolerance(ref, bound, dtype, d, max(lens + [1]), vtop)
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((out.double() - ref).abs() / tol).nan_to_num(nan=9e9).max()))


@pytest.mark.parametrize("form", list(h.FORMS.values()), ids=list(h.FORMS))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
def test_head_dims(nplib, d, dtype, form):
    _compare(nplib, dtype, form, d, 2, 4, 16, [1, 15, 16, 17, 100, 333], seed=d)


@pytest.mark.parametrize("g,ql", [(1, 1), (3, 1), (5, 1), (8, 1), (9, 1), (16, 1), (4, 4), (2, 3), (1, 16), (5, 3)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_groups_and_query_tokens_bf16(nplib, g, ql, d):
    # rows with fewer positions than query tokens: the first ones see nothing
    _compare(nplib, BF16, torch.float8_e4m3fn, d, 2, g, 16, [ql, ql + 1, 0, 1, 40, 700], ql, seed=g + ql)


@pytest.mark.parametrize("g,ql", [(1, 1), (8, 1), (2, 4), (3, 2), (1, 8)])
@pytest.mark.parametrize("d", [16, 128])
def test_groups_and_query_tokens_f32(nplib, g, ql, d):
    _compare(nplib, F32, torch.int8, d, 2, g, 16, [ql, ql + 1, 0, 1, 40, 700], ql, seed=g + ql)


@pytest.mark.parametrize("bs", [1, 2, 3, 5, 8, 24, 32, 64, 100])
@pytest.mark.parametrize("form", list(h.FORMS.values()), ids=list(h.FORMS))
def test_block_sizes(nplib, bs, form):
    _compare(nplib, BF16, form, 128, 4, 2, bs, [1, bs, bs + 1, 37, 5 * bs - 1, 257], seed=bs)


@pytest.mark.parametrize("hk", [1, 2, 3, 4, 5, 6, 7, 8, 11, 12, 16, 24])
@pytest.mark.parametrize("d,g", [(64, 2), (128, 12)])
def test_kv_heads(nplib, hk, d, g):
    _compare(nplib, BF16, torch.float8_e4m3fn, d, hk, g, 16, [300, 1, 0, 77, 1200], seed=hk)


@pytest.mark.parametrize("hk", [1, 3, 4, 5, 8, 10])
def test_kv_heads_wide(nplib, hk):
    """Four warps a block at head_dim 256 with more than eight rows a head: fewer heads a block."""
    _compare(nplib, BF16, torch.int8, 256, hk, 16, 16, [300, 1, 0, 77], seed=hk)
    _compare(nplib, F32, torch.float8_e4m3fn, 256, hk, 4, 16, [300, 1, 0, 77], 2, seed=hk)


def test_fp32_with_long_tables(nplib):
    """Tables that may hold long rows take the kernel that adds each chunk's sum with rounding."""
    rows = [(1, c) for c in (3000, 17, 0, 20000)]
    for d, form in ((128, torch.float8_e4m3fn), (32, torch.int8)):
        inp = h.read_inputs(F32, form, d, 2, 4, 16, rows, cap=200000)
        out, err = _read(nplib, inp, rows, 0.05, 1)
        ref, bound = chunk_reference(h.as_values(inp), rows, 0.05)
        vtop = float(inp["v_scale"].nan_to_num(0, 0).max()) * h.QMAX[form]
        tol = h.decode_tolerance(ref, bound, F32, d, 20000, vtop)
        assert err == 0 and ((out.double() - ref).abs() <= tol).all()
        # far below the bound, which adds up every rounding at its worst: as near as fp32 sums are
        assert float((out.double() - ref).norm() / bound[0].norm()) < 2.0 ** -20


def test_captured_and_replayed(nplib):
    """A process' later calls in a graph: lengths and tables change between replays."""
    rows = [(1, c) for c in (900, 3, 64, 0, 2222)]
    inp = h.read_inputs(BF16, torch.int8, 128, 4, 4, 16, rows)
    ws, out = nplib.decode_q8_workspace(128), torch.zeros_like(inp["q"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nplib.np_paged_decode_q8(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["k_scale"], inp["v_scale"],
                                 inp["block_tables"], inp["context_lens"], 0.1, ws)
    for lens in ([c for _, c in rows], [16, 1, 0, 5, 2000], [0, 0, 0, 0, 0]):
        lens = [min(a, c) for a, (_, c) in zip(lens, rows)]
        inp["context_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        want, _ = _read(nplib, inp, rows, 0.1, 1)
        assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("hk", [1, 8])
def test_one_long_row(nplib, dtype, hk):
    """One row cut over every block of the grid."""
    _compare(nplib, dtype, torch.float8_e4m3fn, 128, hk, 2, 16, [20011], seed=3)


def test_many_rows(nplib):
    """More rows than blocks: most are whole, some cut; rows without history between."""
    gen = torch.Generator().manual_seed(5)
    lens = [int(x) for x in torch.randint(0, 90, (1500,), generator=gen)]
    _compare(nplib, BF16, torch.int8, 32, 2, 2, 8, lens, seed=5)


def test_all_rows_empty(nplib):
    _compare(nplib, BF16, torch.int8, 128, 2, 2, 16, [0, 0, 0])


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-20, 3.0])
def test_scales_of_any_sign(nplib, scale):
    _compare(nplib, BF16, torch.float8_e4m3fn, 64, 2, 4, 16, [5, 200, 64], seed=9, scale=scale)


def test_blocks_of_very_different_scales(nplib):
    """A weight's exponent takes V's scale in: blocks 2^40 apart."""
    _compare(nplib, BF16, torch.float8_e4m3fn, 64, 2, 4, 16, [200, 64], seed=11, scale=1e-9, spread=20)
    _compare(nplib, F32, torch.int8, 64, 2, 4, 16, [200, 64], seed=12, scale=1e-9, spread=20)


def test_zero_and_wild_scales_count_as_their_exponent(nplib):
    inp = h.read_inputs(BF16, torch.float8_e4m3fn, 64, 1, 2, 16, [(1, 64)])
    t = inp["block_tables"][0].long()
    same = dict(inp, k_scale=inp["k_scale"].clone(), v_scale=inp["v_scale"].clone())
    inp["k_scale"][t[0], 0], same["k_scale"][t[0], 0] = 0.0, 2.0 ** -60
    inp["v_scale"][t[1], 0], same["v_scale"][t[1], 0] = 3.7e-3, 2.0 ** -9
    inp["v_scale"][t[2], 0], same["v_scale"][t[2], 0] = -1e-30, 2.0 ** -60
    a, _ = _read(nplib, inp, [(1, 64)], 0.1, 1)
    b, _ = _read(nplib, same, [(1, 64)], 0.1, 1)
    assert torch.equal(a, b)


def test_q_of_any_size(nplib):
    """Rows of q whose elements lie 2^100 apart; a row of zeros."""
    rows = [(1, 50), (1, 50), (1, 50)]
    inp = h.read_inputs(BF16, torch.float8_e4m3fn, 64, 1, 1, 16, rows)
    inp["q"][0] *= 2.0 ** 60
    inp["q"][1] *= 2.0 ** -100
    inp["q"][2] = 0
    for r, scale in ((0, 2.0 ** -60), (1, 2.0 ** 100), (2, 1.0)):
        one = dict(inp, q=inp["q"][r:r + 1], block_tables=inp["block_tables"][r:r + 1].contiguous(),
                   context_lens=inp["context_lens"][r:r + 1], query_starts=inp["query_starts"][:2])
        out, _ = _read(nplib, one, rows[:1], 0.1 * scale, 1)
        ref, bound = chunk_reference(h.as_values(one), rows[:1], 0.1 * scale)
        tol = h.decode_tolerance(ref, bound, BF16, 64, 50, float(inp["v_scale"].nan_to_num(0, 0).max()) * 448)
        assert ((out.double() - ref).abs() <= tol).all()


def test_bad_pages_and_contexts_are_flagged(nplib):
    rows = [(1, 40), (1, 33), (1, 20)]
    inp = h.read_inputs(BF16, torch.int8, 64, 2, 2, 16, rows)
    nb = inp["k_pool"].shape[0]
    inp["block_tables"][0, 1] = nb  # block 0 is read instead
    inp["block_tables"][1, 0] = -5
    _, err = _read(nplib, inp, rows, 0.1, 1)
    assert err == nplib.NP_FLAG_BLOCK_ID
    inp["block_tables"][0, 1] = inp["block_tables"][1, 0] = 0
    inp["context_lens"][2] = -3
    out, err = _read(nplib, inp, rows, 0.1, 1)
    assert err == nplib.NP_FLAG_CONTEXT and (out[2] == 0).all()
    inp["context_lens"][2] = 0
    inp["context_lens"][0] = 16 * inp["block_tables"].shape[1] + 9
    inp["block_tables"][0] = inp["block_tables"][0].clamp(min=0)
    _, err = _read(nplib, inp, rows, 0.1, 1)
    assert err == nplib.NP_FLAG_CONTEXT


def test_same_call_same_bits_and_a_stream_of_its_own(nplib):
    rows = [(1, c) for c in (1000, 3, 64, 700, 2222)]
    inp = h.read_inputs(BF16, torch.float8_e4m3fn, 128, 4, 4, 16, rows)
    a, _ = _read(nplib, inp, rows, 0.1, 1)
    b, _ = _read(nplib, inp, rows, 0.1, 1, stream=torch.cuda.Stream())
    assert torch.equal(a, b)


def test_offsets_past_32_bits(nplib):
    """A pool of more than 2^32 bytes, its last blocks read."""
    nb, bs, hk, d = (1 << 32) // (32 * 8 * 128) + 70, 32, 8, 128
    kp, vp = (torch.zeros(nb, bs, hk, d, dtype=torch.uint8, device="cuda").view(torch.int8) for _ in range(2))
    small = h.read_inputs(BF16, torch.int8, d, hk, 4, bs, [(1, 1000)])
    n = small["k_pool"].shape[0]
    ks, vs = (torch.zeros(nb, hk, device="cuda") for _ in range(2))
    for big, name in ((kp, "k_pool"), (vp, "v_pool"), (ks, "k_scale"), (vs, "v_scale")):
        big[nb - n:] = small[name]
    a, _ = _read(nplib, small, [(1, 1000)], 0.1, 1)
    far = dict(small, k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, block_tables=small["block_tables"] + (nb - n))
    b, err = _read(nplib, far, [(1, 1000)], 0.1, 1)
    assert err == 0 and torch.equal(a, b)
