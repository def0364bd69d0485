"""np_paged_prefill on the GPU against a plain implementation in 64 bits."""
import random

import pytest
import torch

from prompt_helpers import chunk_inputs, chunk_reference, chunk_tolerance

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _run(npg, inp, scale, out=None, ws=None, err=None, stream=None):
    out = torch.full_like(inp["q"], 77.0) if out is None else out
    ws = npg.prefill_workspace(inp["q"].shape[2]) if ws is None else ws
    npg.np_paged_prefill(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["block_tables"],
                         inp["context_lens"], inp["query_starts"], scale, ws, err_word=err,
                         stream=stream)
    return out


def _check(npg, dtype, d, hk, g, bs, rows, scale=None, **kw):
    scale = d ** -0.5 if scale is None else scale
    inp = chunk_inputs(dtype, d, hk, g, bs, rows, **kw)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(npg, inp, scale, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    ref, bound = chunk_reference(inp, rows, scale)
    inside = ~ref.isnan().all(-1).all(-1)
    assert (out[~inside] == 77.0).all()  # tokens of no row are left as they were
    got, ref = out[inside].double(), ref[inside]
    assert got.isfinite().all()
    tol = chunk_tolerance(ref, tuple(b[inside] for b in bound), dtype, d,
                          max([1] + [c for _, c in rows]))
    off = (got - ref).abs()
    assert (off <= tol).all(), f"worst {(off / tol).max().item():.2f} of the tolerance"
    if ref.numel() and ref.norm() > 0:
        # all errors are independent roundings, so their norm is far below the sum of the bounds:
        # bf16, two roundings of 2^-9 sqrt(1/3) each of values no larger than sum p |v|
        rel = (off.norm() / bound[0][inside].norm()).item()
        assert rel < (2.0 ** -8 if dtype == BF else 2e-6), rel
    return inp, out


MIX = [(5, 5), (1, 300), (0, 40), (130, 700), (64, 64), (33, 1000), (2, 2), (257, 257)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("bs", [16, 5])
def test_head_dims(nplib, dtype, d, bs):
    _check(nplib, dtype, d, 2, 4, bs, MIX, before=3, behind=70, seed=d + bs)


@pytest.mark.parametrize("dtype,g", [(BF, g) for g in (1, 2, 3, 5, 6, 7, 8, 12, 16)] +
                         [(F32, g) for g in (1, 2, 3, 5, 7, 8)])
def test_groups(nplib, dtype, g):
    _check(nplib, dtype, 128, 1, g, 16, [(7, 7), (150, 420), (1, 999), (70, 100)], seed=g)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bs", [1, 2, 3, 8, 24, 32, 48, 64, 100, 128, 256, 1000])
def test_block_sizes(nplib, dtype, bs):
    _check(nplib, dtype, 128, 2, 2, bs, [(40, 129), (1, 127), (140, 380), (3, 3)], seed=bs, behind=1)


@pytest.mark.parametrize("hk", [1, 3, 8, 11])
def test_kv_heads(nplib, hk):
    _check(nplib, BF, 64, hk, 2, 16, [(50, 200), (9, 9)], seed=hk)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_tile_edges(nplib, dtype, c):
    rows = [(n, c) for n in sorted({1, c, max(1, c - 1), max(1, c // 2)})]
    _check(nplib, dtype, 128, 1, 2, 16, rows, seed=c)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_see_nothing(nplib, dtype):
    # chunks longer than their context: the first n - c tokens see nothing and get zeros
    rows = [(5, 0), (300, 10), (1, 0), (200, 150), (0, 0), (64, 63)]
    inp, out = _check(nplib, dtype, 64, 2, 3, 8, rows, seed=1)
    assert (out[:5] == 0).all() and (out[5:5 + 290] == 0).all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 256), (BF, 32), (F32, 128)])
@pytest.mark.parametrize("rows", [[(1, 20000)], [(40, 9000)], [(3, 5000), (1, 12000), (300, 300)]])
def test_long_histories_cut_into_many_pieces(nplib, dtype, d, rows):
    _check(nplib, dtype, d, 2, 4, 16, rows, seed=sum(c for _, c in rows) + d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-6, 1.0])
def test_scales(nplib, dtype, scale):
    _check(nplib, dtype, 64, 2, 2, 16, [(20, 90), (130, 130)], scale=scale, seed=4)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 256), (BF, 16), (F32, 64)])
def test_large_scores_move_the_maximum(nplib, dtype, d):
    # keys grow with their position, so the running maximum is replaced again and again
    rows = [(70, 1500), (1, 1400)]
    inp = chunk_inputs(dtype, d, 2, 4, 16, rows, seed=9)
    for r, (_, c) in enumerate(rows):
        t = torch.arange(c, device="cuda")
        b, o = inp["block_tables"][r].long()[t // 16], t % 16
        inp["k_pool"][b, o] = (inp["k_pool"][b, o].float() * (1 + t.float()[:, None, None] / 300)).to(dtype)
    scale = d ** -0.5
    out = _run(nplib, inp, scale)
    torch.cuda.synchronize()
    ref, bound = chunk_reference(inp, rows, scale)
    tol = chunk_tolerance(ref, bound, dtype, d, 1500)
    assert ((out.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("seed", range(24))
def test_random(nplib, seed):
    rnd = random.Random(seed)
    dtype = rnd.choice([BF, BF, F32])
    d = rnd.choice([16, 32, 64, 128, 128, 256])
    g = rnd.choice([1, 2, 3, 4, 5, 7, 8] + ([10, 13, 16] if dtype == BF else []))
    rows = []
    for _ in range(rnd.randint(1, 9)):
        n = rnd.choice([0, 1, 1, rnd.randint(1, 30), rnd.randint(1, 400)])
        rows.append((n, rnd.choice([n, n + rnd.randint(0, 900), rnd.randint(0, n + 5)])))
    _check(nplib, dtype, d, rnd.choice([1, 2, 3, 4, 8]), g, rnd.choice([1, 3, 8, 16, 16, 24, 32, 128]),
           rows, seed=seed, before=rnd.choice([0, 5]), behind=rnd.choice([0, 1, 200]))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 256), (F32, 64)])
def test_one_token_rows_match_the_decode_read(nplib, dtype, d):
    rows = [(1, c) for c in (1, 17, 300, 1024, 2500)]
    inp, out = _check(nplib, dtype, d, 8, 4, 16, rows, seed=2)
    ws = nplib.workspace(5, 32, d, 4)
    dec = torch.empty_like(out)
    nplib.np_paged_decode(None, inp["q"], inp["k_pool"], inp["v_pool"], inp["block_tables"],
                          inp["context_lens"], d ** -0.5, num_splits=4, workspace=ws)
    nplib.np_paged_decode_reduce(dec, ws, 4)
    torch.cuda.synchronize()
    # each is within the tolerance of the same 64-bit values
    ref, bound = chunk_reference(inp, rows, d ** -0.5)
    tol = chunk_tolerance(ref, bound, dtype, d, 2500)
    assert ((out.double() - dec.double()).abs() <= 2 * tol).all()


@pytest.mark.parametrize("dtype,d,g", [(BF, 128, 4), (BF, 64, 1), (BF, 16, 8), (BF, 256, 4), (F32, 64, 2)])
def test_mixed_batches(nplib, dtype, d, g):
    """Many one-token rows among chunks: a block passes again and again from units of one tile to
    units of two, a dozen kv tiles each."""
    rnd = random.Random(d)
    rows = [(1, rnd.randint(200, 2500)) for _ in range(40)] + [(300, 1500), (513, 800), (300, 300)]
    rnd.shuffle(rows)
    _check(nplib, dtype, d, 8, g, 16, rows, seed=d + g)


def test_no_rows_and_no_tokens(nplib):
    inp = chunk_inputs(BF, 64, 1, 2, 16, [(4, 4)])
    out = torch.full_like(inp["q"], 5.0)
    ws = nplib.prefill_workspace(64)
    a = (inp["k_pool"], inp["v_pool"])
    nplib.np_paged_prefill(out, inp["q"], *a, inp["block_tables"][:0], inp["context_lens"][:0],
                           inp["query_starts"][:1], 0.1, ws)
    e = inp["q"][:0]
    nplib.np_paged_prefill(e.clone(), e, *a, inp["block_tables"], inp["context_lens"],
                           inp["query_starts"] * 0, 0.1, ws)
    nplib.np_paged_prefill(out, inp["q"], *a, inp["block_tables"], inp["context_lens"],
                           inp["query_starts"] * 0, 0.1, ws)  # rows without tokens
    torch.cuda.synchronize()
    assert (out == 5.0).all()


def test_many_rows(nplib):
    rows = [(1 + r % 3, 5 + (r * 37) % 200) for r in range(1500)]
    _check(nplib, BF, 64, 1, 2, 16, rows, seed=3)
    _check(nplib, F32, 16, 1, 1, 8, [(r % 2, r % 2 + r % 5) for r in range(4096)], seed=4)


@pytest.mark.parametrize("dtype,d,bs", [(BF, 128, 16), (BF, 64, 5), (F32, 64, 16)])
def test_bad_metadata_is_flagged_and_stays_in_bounds(nplib, dtype, d, bs):
    rows = [(20, 100), (30, 200), (1, 50)]

    def flags(change):
        inp = chunk_inputs(dtype, d, 2, 2, bs, rows, seed=6, poison=False)
        change(inp)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = _run(nplib, inp, 0.1, err=err)
        torch.cuda.synchronize()
        return int(err), out, inp

    def set_(key, i, v):
        def f(inp):
            inp[key][i] = v
        return f

    nb = sum(-(-c // bs) for _, c in rows) + 3
    clean = flags(lambda inp: None)
    assert clean[0] == 0
    e, out, inp = flags(set_("block_tables", (1, 2), nb))
    assert e == nplib.NP_FLAG_BLOCK_ID
    assert torch.equal(out[:20], clean[1][:20]) and torch.equal(out[50:], clean[1][50:])
    # block 0 stands in for it
    want = flags(set_("block_tables", (1, 2), 0))
    assert want[0] == 0 and torch.equal(out, want[1])
    assert flags(set_("block_tables", (0, 0), -5))[0] == nplib.NP_FLAG_BLOCK_ID
    assert flags(set_("context_lens", 2, -3))[0] == nplib.NP_FLAG_CONTEXT
    assert (flags(set_("context_lens", 2, -3))[1][50] == 0).all()
    cap = clean[2]["block_tables"].shape[1] * bs
    e, out, _ = flags(lambda inp: (set_("block_tables", 2, 1)(inp), set_("context_lens", 2, cap + 1)(inp)))
    assert e == nplib.NP_FLAG_CONTEXT
    # the other rows' values are the same sums; the shares' ends move with the batch's lengths, so
    # each is within the tolerance of the exact value and not the same bits
    ref, bound = chunk_reference(clean[2], rows, 0.1)
    tol = chunk_tolerance(ref, bound, dtype, d, 200)
    assert ((out.double() - ref).abs() <= tol)[:50].all()
    for v in (-1, 10, 10 ** 9):
        assert flags(set_("query_starts", 2, v))[0] == nplib.NP_FLAG_QUERY
    assert flags(set_("query_starts", 3, 60))[0] == nplib.NP_FLAG_QUERY
    assert flags(set_("query_starts", 0, -7))[0] == nplib.NP_FLAG_QUERY


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 256), (F32, 128)])
def test_same_bits_every_time_on_any_stream_and_in_graphs(nplib, dtype, d):
    rows = [(200, 900), (1, 4000), (33, 33)]
    inp, want = _check(nplib, dtype, d, 2, 4, 16, rows, seed=8)
    for _ in range(3):
        assert torch.equal(_run(nplib, inp, d ** -0.5, out=torch.zeros_like(want)), want + 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _run(nplib, inp, d ** -0.5, out=torch.zeros_like(want), stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    # two graphs, each with its workspace, replayed next to each other
    outs = [torch.zeros_like(want) for _ in range(2)]
    ws = [nplib.prefill_workspace(d).fill_(255) for _ in range(2)]
    graphs = []
    for o, w in zip(outs, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _run(nplib, inp, d ** -0.5, out=o, ws=w)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    # lengths are read on the device: a replay after they change gives the new answer
    inp["context_lens"][1] = 77
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    ref, bound = chunk_reference(inp, [(200, 900), (1, 77), (33, 33)], d ** -0.5)
    assert ((outs[0].double() - ref).abs() <= chunk_tolerance(ref, bound, dtype, d, 900)).all()


@pytest.mark.parametrize("a,b", [((BF, 32), (F32, 16)), ((BF, 16), (F32, 32)), ((F32, 16), (F32, 16)),
                                 ((BF, 128), (F32, 64)), ((BF, 256), (F32, 256))])
def test_two_different_calls_at_once(nplib, a, b):
    # narrow heads leave room on an SM for a block of each call: both want its tensor memory
    rows = [(300, 900), (1, 2000), (65, 65)]
    calls = [_check(nplib, dtype, d, 4, 4, 16, rows, seed=9 + i) for i, (dtype, d) in enumerate((a, b))]
    outs = [torch.zeros_like(want) for _, want in calls]
    ws = [nplib.prefill_workspace(inp["q"].shape[2]).fill_(255) for inp, _ in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for o in outs:
        o.fill_(77.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for (inp, _), o, w, st in zip(calls, outs, ws, streams):
            _run(nplib, inp, inp["q"].shape[2] ** -0.5, out=o, ws=w, stream=st)
    torch.cuda.synchronize()
    for (_, want), o in zip(calls, outs):
        assert torch.equal(o, want)


@pytest.mark.parametrize("dtype,hk,d,bs", [(BF, 8, 128, 16), (BF, 8, 128, 7), (F32, 8, 128, 16)])
def test_pool_offsets_past_32_bits(nplib, dtype, hk, d, bs):
    nb = (2 ** 31 // (hk * d) + 8192) // bs  # more than 2^31 elements
    rows = [(20, 300)]
    small = chunk_inputs(dtype, d, hk, 2, bs, rows, seed=10, poison=False)
    want = _run(nplib, small, 0.1)
    n = small["k_pool"].shape[0]
    big = dict(small)
    for key in ("k_pool", "v_pool"):
        big[key] = torch.zeros(nb, bs, hk, d, dtype=dtype, device="cuda")
        big[key][nb - n:] = small[key]
    big["block_tables"] = small["block_tables"] + (nb - n)
    got = _run(nplib, big, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", [False, True])
def test_a_prompt_in_chunks_then_decode(nplib, dtype, norm):
    """A row's prompt as it is served: two chunks through prefill_step, then decode steps whose new
    token np_rope_append rotates into the cache; every output against one causal attention of
    all tokens in 64 bits over the rotated values the pools hold."""
    hq, hk, d, bs, lens, steps = 8, 2, 128, 16, (50, 33), 3
    total = sum(lens) + steps
    gen = torch.Generator().manual_seed(11)
    x = [torch.randn(total, h, d, generator=gen).to(dtype).cuda() for h in (hq, hk, hk)]
    w = [(1 + 0.1 * torch.randn(d, generator=gen)).to(dtype).cuda() if norm else None for _ in range(2)]
    table = nplib.rope_table(256, d)
    nblk = -(-total // bs)
    ids = torch.randperm(nblk + 2, generator=gen)[:nblk].to(torch.int32).cuda()
    kp = torch.full((nblk + 2, bs, hk, d), float("nan"), dtype=dtype, device="cuda")
    vp = kp.clone()
    t = torch.arange(total, device="cuda")
    slots = ids[t // bs].long() * bs + t % bs
    pos = t.to(torch.int32)
    ws = nplib.prefill_workspace(d)
    q_rot, outs = torch.empty_like(x[0]), torch.empty_like(x[0])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = 0
    for n in lens:
        s = slice(at, at + n)
        nplib.prefill_step(outs[s], x[0][s], x[1][s], x[2][s], slots[s], kp, vp, ids[None],
                           torch.tensor([at + n], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, n], dtype=torch.int32, device="cuda"), d ** -0.5, ws,
                           cos_sin=table, positions=pos[s], q_weight=w[0], k_weight=w[1],
                           q_rotated=q_rot[s], err_word=err)
        at += n
    for _ in range(steps):
        s = slice(at, at + 1)
        nplib.np_rope_append(q_rot[s], x[0][s], x[1][s], x[2][s], slots[s], kp, vp, table, pos[s],
                             q_weight=w[0], k_weight=w[1], err_word=err)
        S = nplib.np_paged_decode_plan(1, hq, hk, d, bs, nblk, dtype)
        nplib.decode_step(outs[s], q_rot[s], kp, vp, ids[None],
                          torch.tensor([at + 1], dtype=torch.int32, device="cuda"), d ** -0.5,
                          num_splits=S, workspace=nplib.workspace(1, hq, d, S), err_word=err)
        at += 1
    torch.cuda.synchronize()
    assert int(err) == 0
    inp = dict(q=q_rot, k_pool=kp, v_pool=vp, block_tables=ids[None],
               query_starts=torch.tensor([0, total], dtype=torch.int32, device="cuda"))
    ref, bound = chunk_reference(inp, [(total, total)], d ** -0.5)
    assert ((outs.double() - ref).abs() <= chunk_tolerance(ref, bound, dtype, d, total)).all()


def test_prefill_step_without_rotation(nplib):
    rows = [(30, 30), (5, 90)]
    inp, want = _check(nplib, BF, 64, 2, 2, 16, rows, seed=12)
    # the chunk's own K and V, taken out of the pools and appended again
    new = []
    for r, (n, c) in enumerate(rows):
        t = torch.arange(c - n, c, device="cuda")
        new.append(inp["block_tables"][r].long()[t // 16] * 16 + t % 16)
    slots = torch.cat(new)
    k, v = (inp[x].view(-1, 2, 64)[slots].clone() for x in ("k_pool", "v_pool"))
    for x in ("k_pool", "v_pool"):
        inp[x].view(-1, 2, 64)[slots] = float("nan")
    out = torch.full_like(want, 77.0)
    nplib.prefill_step(out, inp["q"], k, v, slots, inp["k_pool"], inp["v_pool"], inp["block_tables"],
                       inp["context_lens"], inp["query_starts"], 64 ** -0.5, nplib.prefill_workspace(64))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_tensor_of_another_device_or_on_the_host_is_refused(nplib):
    inp = chunk_inputs(BF, 64, 1, 2, 16, [(4, 4)])
    ws = nplib.prefill_workspace(64)
    with pytest.raises(ValueError, match="CUDA"):
        nplib.np_paged_prefill(torch.empty_like(inp["q"]), inp["q"].cpu(), inp["k_pool"], inp["v_pool"],
                               inp["block_tables"], inp["context_lens"], inp["query_starts"], 0.1, ws)
    with pytest.raises(nplib.NPError, match="WORKSPACE"):
        nplib.np_paged_prefill(torch.empty_like(inp["q"]), inp["q"], inp["k_pool"], inp["v_pool"],
                               inp["block_tables"], inp["context_lens"], inp["query_starts"], 0.1,
                               ws[:1024])
    with pytest.raises(nplib.NPError, match="INVALID"):
        _run(nplib, inp, 0.1, out=inp["q"])
