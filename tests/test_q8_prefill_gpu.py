"""np_paged_prefill_q8 against the formula in 64 bits."""
import pytest
import torch

import q8_helpers as h
from prompt_helpers import chunk_reference

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def _run(npg, inp, scale, stream=None, **kw):
    out, ws = torch.full_like(inp["q"], 77.0), npg.prefill_workspace(inp["q"].shape[2])
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    npg.np_paged_prefill_q8(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["k_scale"], inp["v_scale"],
                            inp["block_tables"], inp["context_lens"], inp["query_starts"], scale, ws,
                            stream=stream, **kw)
    torch.cuda.synchronize()
    return out


def _check(npg, dtype, form, d, hk, g, bs, rows, scale=None, **kw):
    scale = d ** -0.5 / 2 if scale is None else scale
    inp = h.read_inputs(dtype, form, d, hk, g, bs, rows, **kw)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(npg, inp, scale, err_word=err)
    assert int(err) == 0
    ref, bound = chunk_reference(h.as_values(inp), rows, scale)
    inside = ~ref.isnan().all(-1).all(-1)
    assert (out[~inside] == 77.0).all()  # tokens of no row are left as they were
    got, ref = out[inside].double(), ref[inside]
    assert got.isfinite().all()
    tol = h.prefill_tolerance(inp, ref, tuple(b[inside] for b in bound), dtype, d, max([1] + [c for _, c in rows]),
                              scale)
    off = (got - ref).abs()
    assert (off <= tol).all(), f"worst {(off / tol).max().item():.2f} of the tolerance"
    return inp, out


MIX = [(5, 5), (1, 300), (0, 40), (130, 700), (64, 64), (33, 1000), (2, 2), (257, 257)]


@pytest.mark.parametrize("form", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("bs", [16, 5])
def test_head_dims(nplib, dtype, form, d, bs):
    _check(nplib, dtype, form, d, 2, 4, bs, MIX, before=3, behind=70, seed=d + bs)


@pytest.mark.parametrize("dtype,g", [(BF, g) for g in (1, 2, 3, 5, 8, 12, 16)] + [(F32, g) for g in (1, 3, 7, 8)])
def test_groups(nplib, dtype, g):
    _check(nplib, dtype, E4M3, 128, 1, g, 16, [(7, 7), (150, 420), (1, 999), (70, 100)], seed=g)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bs", [1, 2, 3, 8, 24, 32, 64, 100, 128, 256, 1000])
def test_block_sizes(nplib, dtype, bs):
    _check(nplib, dtype, INT8, 128, 2, 2, bs, [(40, 129), (1, 127), (140, 380), (3, 3)], seed=bs, behind=1)


@pytest.mark.parametrize("hk", [1, 3, 8, 11])
def test_kv_heads(nplib, hk):
    _check(nplib, BF, E4M3, 64, hk, 2, 16, [(50, 200), (9, 9)], seed=hk)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("c", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_tile_edges(nplib, dtype, c):
    rows = [(n, c) for n in sorted({1, c, max(1, c - 1), max(1, c // 2)})]
    _check(nplib, dtype, E4M3, 128, 1, 2, 16, rows, seed=c)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rows_that_see_nothing(nplib, dtype):
    rows = [(5, 0), (300, 10), (1, 0), (200, 150), (0, 0), (64, 63)]
    inp, out = _check(nplib, dtype, INT8, 64, 2, 3, 8, rows, seed=1)
    assert (out[:5] == 0).all() and (out[5:5 + 290] == 0).all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 256), (BF, 32), (F32, 128)])
@pytest.mark.parametrize("rows", [[(1, 20000)], [(40, 9000)], [(3, 5000), (1, 12000), (300, 300)]])
def test_long_histories_cut_into_many_pieces(nplib, dtype, d, rows):
    _check(nplib, dtype, E4M3, d, 2, 4, 16, rows, seed=sum(c for _, c in rows) + d)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-6, 1.0])
def test_scales(nplib, dtype, form, scale):
    _check(nplib, dtype, form, 64, 2, 2, 16, [(20, 90), (130, 130)], scale=scale, seed=4)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_scales_of_blocks_of_any_size(nplib, dtype):
    """Blocks 2^40 apart, and ones whose scale is at either end."""
    _check(nplib, dtype, E4M3, 128, 2, 4, 16, [(40, 200), (64, 64)], seed=11, scale=1e-9, spread=20)
    inp = h.read_inputs(dtype, INT8, 64, 1, 2, 16, [(30, 64)])
    t = inp["block_tables"][0].long()
    inp["k_scale"][t[0], 0], inp["v_scale"][t[1], 0], inp["v_scale"][t[2], 0] = 0.0, 2.0 ** 60, -3.0
    same = dict(inp, k_scale=inp["k_scale"].clone(), v_scale=inp["v_scale"].clone())
    same["k_scale"][t[0], 0], same["v_scale"][t[2], 0] = 2.0 ** -60, 2.0
    assert torch.equal(_run(nplib, inp, 0.1), _run(nplib, same, 0.1))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("e", [-60, -5, 0, 7, 8, 60])
def test_every_code_under_small_and_large_scales(nplib, form, dtype, e):
    """One position a row, so that its V comes out as it is: a weight over itself (as the two fp16
    parts of the decode read's kernel, 2^-22 off, where q is fp32; l and the quotient rounded)."""
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    skip = codes == 0x80 if form is INT8 else (codes & 0x7f) == 0x7f
    codes = torch.where(skip, torch.zeros_like(codes), codes)
    d = 64
    v = codes.view(4, 1, 1, d).view(form).cuda()
    q = torch.ones(4, 1, d, dtype=dtype, device="cuda")
    scale = torch.full((4, 1), 2.0 ** e, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    inp = dict(q=q, k_pool=v, v_pool=v, k_scale=torch.ones_like(scale), v_scale=scale,
               block_tables=torch.arange(4, **i32)[:, None].contiguous(), context_lens=torch.ones(4, **i32),
               query_starts=torch.arange(5, **i32))
    out = _run(nplib, inp, 0.01)
    want = v.float().double().flatten() * 2.0 ** e
    off = (out.double().flatten() - want).abs()
    assert (off <= want.abs() * (0.0 if dtype is BF else 2.0 ** -22 + 3 * 2.0 ** -24)).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("bs", [1, 16])
def test_every_code_exactly(nplib, form, dtype, n, bs):
    """As above with keys of zero, so that the weight is a power of two: in every way that V comes (the
    first n - 1 tokens see nothing)."""
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    skip = codes == 0x80 if form is INT8 else (codes & 0x7f) == 0x7f
    codes = torch.where(skip, torch.zeros_like(codes), codes)
    d = 64
    v = torch.full((4, bs, 1, d), 0x7f if form is E4M3 else 0x80, dtype=torch.uint8)
    v[:, 0] = codes.view(4, 1, d)
    v = v.view(form).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    scale = torch.tensor([[2.0 ** -60], [2.0 ** -3], [2.0 ** 9], [2.0 ** 60]], device="cuda")
    inp = dict(q=torch.ones(4 * n, 1, d, dtype=dtype, device="cuda"),
               k_pool=torch.zeros(4, bs, 1, d, dtype=torch.uint8, device="cuda").view(form), v_pool=v,
               k_scale=torch.ones_like(scale), v_scale=scale,
               block_tables=torch.arange(4, **i32)[:, None].contiguous(), context_lens=torch.ones(4, **i32),
               query_starts=torch.arange(5, **i32) * n)
    out = _run(nplib, inp, 0.01).view(4, n, d).double()
    assert torch.equal(out[:, -1], v[:, 0, 0].float().double() * scale.double()) and (out[:, :-1] == 0).all()


def test_many_rows(nplib):
    gen = torch.Generator().manual_seed(2)
    rows = [(1 + int(x) % 3, 3 + int(x)) for x in torch.randint(0, 60, (600,), generator=gen)]
    _check(nplib, BF, INT8, 64, 1, 4, 16, rows, seed=5)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("g", [1, 3, 8, 16])
@pytest.mark.parametrize("d", [32, 128])
def test_short_rows_among_long_ones(nplib, dtype, g, d):
    """Rows whose tokens fit one fetch are another kernel's: every count around that border, with and
    without a history, among chunks; and such rows alone."""
    if g == 16 and dtype is F32:
        g = 7
    rows = [(n, c) for n in (0, 1, 2, 3, 4, 7, 8, 9, 17) for c in (0, 1, n, 100, 1111)]
    _check(nplib, dtype, E4M3, d, 2, g, 16, rows + [(130, 300)], seed=g, before=2, behind=3)
    _check(nplib, dtype, INT8, d, 3, g, 8, [(1, c) for c in (5, 0, 700, 64, 2000)], seed=g, behind=1)
    _check(nplib, dtype, INT8, d, 1, g, 5, [(1, 3000)], seed=g)
    _check(nplib, dtype, INT8, d, 1, g, 16, [(0, 30), (1, 3000), (0, 0)], seed=g)


def test_bad_metadata_is_flagged(nplib):
    rows = [(4, 40), (3, 33), (1, 20)]
    inp = h.read_inputs(BF, E4M3, 128, 2, 2, 16, rows)
    inp["block_tables"][0, 1], inp["block_tables"][1, 0] = inp["k_pool"].shape[0], -5
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _run(nplib, inp, 0.1, err_word=err)
    assert int(err) == nplib.NP_FLAG_BLOCK_ID
    inp["block_tables"][:2] = 0
    inp["context_lens"][2] = -3
    inp["query_starts"][3] = 99
    err.zero_()
    _run(nplib, inp, 0.1, err_word=err)
    assert int(err) == nplib.NP_FLAG_CONTEXT | nplib.NP_FLAG_QUERY


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 256), (BF, 32), (F32, 128), (F32, 256)])
def test_same_bits_every_time_on_any_stream_and_in_graphs(nplib, dtype, d):
    rows = [(200, 900), (1, 2500), (30, 30)]
    inp = h.read_inputs(dtype, E4M3, d, 2, 4, 16, rows, seed=d)
    want = _run(nplib, inp, 0.1)
    assert torch.equal(want, _run(nplib, inp, 0.1, stream=torch.cuda.Stream()))
    ws, out = nplib.prefill_workspace(d), torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nplib.np_paged_prefill_q8(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["k_scale"], inp["v_scale"],
                                  inp["block_tables"], inp["context_lens"], inp["query_starts"], 0.1, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_pool_offsets_past_32_bits(nplib):
    nb, bs, hk, d = (1 << 32) // (32 * 8 * 128) + 70, 32, 8, 128
    kp, vp = (torch.zeros(nb, bs, hk, d, dtype=torch.int8, device="cuda") for _ in range(2))
    rows = [(40, 1000), (1, 300)]
    small = h.read_inputs(BF, INT8, d, hk, 4, bs, rows)
    n = small["k_pool"].shape[0]
    ks, vs = (torch.zeros(nb, hk, device="cuda") for _ in range(2))
    for big, name in ((kp, "k_pool"), (vp, "v_pool"), (ks, "k_scale"), (vs, "v_scale")):
        big[nb - n:] = small[name]
    far = dict(small, k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, block_tables=small["block_tables"] + (nb - n))
    assert torch.equal(_run(nplib, small, 0.1), _run(nplib, far, 0.1))
