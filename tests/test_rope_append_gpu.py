"""np_rope_append on the GPU against a plain implementation in 64 bits."""
import pytest
import torch

from prompt_helpers import rope_reference, rope_tolerance

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _case(dtype, t, hq, hk, d, rot, *, axes=1, sections=None, norm=False, fused=False, bs=16, seed=0,
          max_pos=1000):
    g = torch.Generator().manual_seed(seed)
    if fused:
        rows = torch.randn(t, (hq + 2 * hk) * d, generator=g).to(dtype).cuda()
        q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split([hq * d, hk * d, hk * d], 1))
    else:
        q, k, v = (torch.randn(t, h, d, generator=g).to(dtype).cuda() for h in (hq, hk, hk))
    nb = -(-t // bs) + 3
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    return dict(
        q=q, k=k, v=v, table=torch.cat([ang.cos(), ang.sin()], 1).float().cuda(),
        pos=torch.randint(0, max_pos, (axes, t) if axes > 1 else (t,), generator=g,
                          dtype=torch.int32).cuda(),
        slots=torch.randperm(nb * bs, generator=g)[:t].cuda(), sections=sections,
        k_pool=torch.randn(nb, bs, hk, d, generator=g).to(dtype).cuda(),
        v_pool=torch.randn(nb, bs, hk, d, generator=g).to(dtype).cuda(),
        qw=(1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() if norm else None,
        kw=(1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() if norm else None)


def _check(npg, c, interleaved=False, eps=1e-6, in_place=False, stream=None):
    dtype, d = c["k"].dtype, c["k"].shape[2]
    t, hk = c["k"].shape[:2]
    (yq, zq), (yk, zk) = rope_reference(c["q"], c["k"], c["table"], c["pos"], c["sections"],
                                        interleaved, c["qw"], c["kw"], eps)
    kp, vp = c["k_pool"].clone(), c["v_pool"].clone()
    q_in = c["q"].clone() if in_place else c["q"]
    q_out = q_in if in_place else torch.full(c["q"].shape, float("nan"), dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    npg.np_rope_append(q_out, q_in, c["k"], c["v"], c["slots"], kp, vp, c["table"], c["pos"],
                       sections=c["sections"], interleaved=interleaved, q_weight=c["qw"],
                       k_weight=c["kw"], eps=eps, err_word=err, stream=stream)
    torch.cuda.synchronize()
    norm = c["qw"] is not None
    assert ((q_out.double() - yq).abs() <= rope_tolerance(yq, zq, dtype, d, norm)).all()
    live = c["slots"] >= 0
    got = kp.view(-1, hk, d)[c["slots"][live]].double()
    assert ((got - yk[live]).abs() <= rope_tolerance(yk, zk, dtype, d, c["kw"] is not None)[live]).all()
    assert torch.equal(vp.view(-1, hk, d)[c["slots"][live]], c["v"][live])
    rest = torch.ones(kp.shape[0] * kp.shape[1], dtype=torch.bool, device="cuda")
    rest[c["slots"][live]] = False
    for new, old in ((kp, c["k_pool"]), (vp, c["v_pool"])):  # every other slot as it was
        assert torch.equal(new.view(-1, hk, d)[rest], old.view(-1, hk, d)[rest])
    assert int(err) == 0
    return q_out, kp, vp


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot", [(16, 16), (32, 32), (64, 64), (64, 32), (128, 128), (128, 48),
                                   (256, 256), (256, 16), (256, 80)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_shapes(nplib, dtype, d, rot, interleaved, norm):
    _check(nplib, _case(dtype, 37, 6, 2, d, rot, norm=norm, fused=norm, seed=d + rot), interleaved)


@pytest.mark.parametrize("t", [1, 2, 31, 257, 2000])
@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 1), (32, 8), (40, 8), (7, 3), (128, 16)])
def test_tokens_and_heads(nplib, t, hq, hk):
    _check(nplib, _case(BF, t, hq, hk, 128, 128, norm=True, fused=t % 2 == 1, bs=8, seed=t + hq))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,hq,hk", [(16, 5, 1), (32, 3, 2), (64, 6, 2), (128, 7, 3), (256, 2, 1)])
@pytest.mark.parametrize("t", [511, 512, 2047, 2048, 2500])
def test_every_block_size(nplib, dtype, d, hq, hk, t):
    # the launcher chooses the block by the number of tokens: both sides of each border, heads that
    # do not fill a block
    _check(nplib, _case(dtype, t, hq, hk, d, d, norm=d != 32, fused=d == 64, seed=t + d), t % 2 == 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes,rot,sections", [(3, 128, (16, 24, 24)), (3, 64, (5, 14, 13)),
                                               (2, 32, (0, 16)), (4, 64, (1, 0, 30, 1)),
                                               (3, 16, (2, 3, 3)), (1, 64, (32,))])
def test_axes(nplib, dtype, interleaved, axes, rot, sections):
    _check(nplib, _case(dtype, 53, 4, 2, 128, rot, axes=axes, sections=sections, norm=True,
                        seed=axes + rot), interleaved)


def test_axes_that_agree_are_one_axis(nplib):
    c = _case(BF, 40, 4, 2, 64, 64, seed=3)
    a = _check(nplib, c)
    c3 = dict(c, pos=c["pos"].expand(3, -1).contiguous(), sections=(8, 12, 12))
    for x, y in zip(a, _check(nplib, c3)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(nplib, dtype):
    c = _case(dtype, 300, 12, 4, 128, 128, norm=True, seed=5)
    a, b = _check(nplib, c)[0], _check(nplib, c, in_place=True)[0]
    assert torch.equal(a, b)


def test_only_one_weight(nplib):
    c = _case(BF, 21, 4, 2, 128, 128, norm=True, seed=6)
    (yq, zq), (yk, zk) = rope_reference(c["q"], c["k"], c["table"], c["pos"], None, False, None,
                                        c["kw"], 1e-6)
    q_out, kp, vp = torch.empty_like(c["q"]), c["k_pool"].clone(), c["v_pool"].clone()
    nplib.np_rope_append(q_out, c["q"], c["k"], c["v"], c["slots"], kp, vp, c["table"], c["pos"],
                         k_weight=c["kw"])
    torch.cuda.synchronize()
    assert ((q_out.double() - yq).abs() <= rope_tolerance(yq, zq, BF, 128, False)).all()
    got = kp.view(-1, 2, 128)[c["slots"]].double()
    assert ((got - yk).abs() <= rope_tolerance(yk, zk, BF, 128, True)).all()


def test_position_zero_and_v_are_bit_exact(nplib):
    c = _case(F32, 9, 2, 2, 64, 64, seed=7)
    c["pos"].zero_()  # the angle is zero: cos 1, sin 0
    q_out, kp, vp = _check(nplib, c)
    assert torch.equal(q_out, c["q"])
    assert torch.equal(kp.view(-1, 2, 64)[c["slots"]], c["k"])


def test_values_that_are_not_finite_stay_in_their_head(nplib):
    c = _case(BF, 8, 4, 2, 128, 128, norm=True, seed=8)
    c["q"][3, 1, 5] = float("nan")
    c["k"][2, 0, 7] = float("inf")
    c["v"][1, 1, 0] = float("nan")
    q_out, kp, vp = torch.empty_like(c["q"]), c["k_pool"].clone(), c["v_pool"].clone()
    nplib.np_rope_append(q_out, c["q"], c["k"], c["v"], c["slots"], kp, vp, c["table"], c["pos"],
                         q_weight=c["qw"], k_weight=c["kw"])
    torch.cuda.synchronize()
    bad = ~q_out.isfinite().all(-1)
    assert bad.nonzero().tolist() == [[3, 1]]
    assert (~kp.view(-1, 2, 128)[c["slots"]].isfinite().all(-1)).nonzero().tolist() == [[2, 0]]
    assert torch.equal(vp.view(-1, 2, 128)[c["slots"]].view(torch.int16), c["v"].view(torch.int16))


def test_zero_rows_stay_zero(nplib):
    c = _case(BF, 5, 2, 1, 32, 32, norm=True, seed=9)
    c["q"].zero_()
    assert (_check(nplib, c)[0] == 0).all()


def test_padding_and_bad_slots(nplib):
    c = _case(BF, 40, 4, 2, 64, 64, seed=10)
    c["slots"][::3] = -1
    _check(nplib, c)  # q of padding tokens is written all the same
    slots = c["slots"].clone()
    slots[1] = c["k_pool"].shape[0] * c["k_pool"].shape[1]  # one past the pool
    slots[2] = 2 ** 40
    kp, vp = c["k_pool"].clone(), c["v_pool"].clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    nplib.np_rope_append(torch.empty_like(c["q"]), c["q"], c["k"], c["v"], slots, kp, vp, c["table"],
                         c["pos"], err_word=err)
    torch.cuda.synchronize()
    assert int(err) == nplib.NP_FLAG_SLOT
    untouched = torch.ones(kp.shape[0] * kp.shape[1], dtype=torch.bool, device="cuda")
    ok = (slots >= 0) & (slots < untouched.numel())
    untouched[slots[ok]] = False
    assert torch.equal(kp.view(-1, 2, 64)[untouched], c["k_pool"].view(-1, 2, 64)[untouched])


@pytest.mark.parametrize("axes", [1, 3])
def test_positions_outside_the_table_are_clamped_and_flagged(nplib, axes):
    c = _case(F32, 12, 2, 1, 64, 64, axes=axes, sections=(8, 12, 12) if axes == 3 else None, seed=11)
    p = c["pos"].view(axes, -1)
    p[0, 3], p[-1, 5], p[0, 7] = -1, c["table"].shape[0], 2 ** 31 - 1
    (yq, zq), _ = rope_reference(c["q"], c["k"], c["table"], c["pos"], c["sections"], False, None,
                                 None, 0.0)
    q_out, err = torch.empty_like(c["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    nplib.np_rope_append(q_out, c["q"], c["k"], c["v"], c["slots"], c["k_pool"].clone(),
                         c["v_pool"].clone(), c["table"], c["pos"], sections=c["sections"],
                         err_word=err)
    torch.cuda.synchronize()
    assert int(err) == nplib.NP_FLAG_POSITION
    assert ((q_out.double() - yq).abs() <= rope_tolerance(yq, zq, F32, 64, False)).all()


def test_keys_and_values_only(nplib):
    c = _case(BF, 30, 4, 2, 128, 128, norm=True, seed=12)
    want = _check(nplib, c)
    kp, vp = c["k_pool"].clone(), c["v_pool"].clone()
    nplib.np_rope_append(None, None, c["k"], c["v"], c["slots"], kp, vp, c["table"], c["pos"],
                         k_weight=c["kw"])
    torch.cuda.synchronize()
    assert torch.equal(kp, want[1]) and torch.equal(vp, want[2])


def test_no_tokens(nplib):
    c = _case(BF, 4, 4, 2, 128, 128, seed=13)
    kp = c["k_pool"].clone()
    e = lambda x: x[:0]  # noqa: E731
    nplib.np_rope_append(e(c["q"]).clone(), e(c["q"]), e(c["k"]), e(c["v"]), e(c["slots"]), kp,
                         c["v_pool"], c["table"], e(c["pos"]))
    torch.cuda.synchronize()
    assert torch.equal(kp, c["k_pool"])


def test_pool_offsets_past_32_bits(nplib):
    hk, d, bs = 8, 128, 16
    nb = (2 ** 31 // (hk * d) + 4096) // bs  # more than 2^31 elements
    c = _case(BF, 20, 4, hk, d, d, seed=14)
    kp = torch.zeros(nb, bs, hk, d, dtype=BF, device="cuda")
    vp = torch.zeros_like(kp)
    slots = nb * bs - 1 - torch.arange(20, device="cuda") * 7
    nplib.np_rope_append(torch.empty_like(c["q"]), c["q"], c["k"], c["v"], slots, kp, vp, c["table"],
                         c["pos"])
    torch.cuda.synchronize()
    _, (yk, zk) = rope_reference(c["q"], c["k"], c["table"], c["pos"], None, False, None, None, 0.0)
    got = kp.view(-1, hk, d)[slots].double()
    assert ((got - yk).abs() <= rope_tolerance(yk, zk, BF, d, False)).all()
    assert torch.equal(vp.view(-1, hk, d)[slots], c["v"])
    assert int(torch.count_nonzero(vp.view(-1, hk * d)[:2 ** 20])) == 0


def test_another_stream_and_a_graph(nplib):
    c = _case(BF, 70, 8, 2, 128, 128, norm=True, fused=True, seed=15)
    want = _check(nplib, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _check(nplib, c, stream=s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    q_out, kp, vp = torch.zeros_like(want[0]), c["k_pool"].clone(), c["v_pool"].clone()
    args = (q_out, c["q"], c["k"], c["v"], c["slots"], kp, vp, c["table"], c["pos"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nplib.np_rope_append(*args, q_weight=c["qw"], k_weight=c["kw"])
    for _ in range(2):
        q_out.zero_()
        kp.copy_(c["k_pool"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, want[0]) and torch.equal(kp, want[1])


def test_rope_table_against_the_formula(nplib):
    t = nplib.rope_table(131072, 64, base=500000.0)
    p = 131071
    ang = p * 500000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    want = torch.cat([ang.cos(), ang.sin()])
    # the angle (up to 131071) is off by 2 x 2^-53 of itself, the function by less than 2^-50, and the
    # value is rounded to fp32
    assert ((t[p].cpu().double() - want).abs() <= 131071 * 2.0 ** -51 + 2.0 ** -24 * want.abs()).all()
    f = torch.linspace(1, 0.01, 32)
    t2 = nplib.rope_table(10, 64, inv_freq=f)
    assert torch.equal(t2[0], torch.cat([torch.ones(32), torch.zeros(32)]).cuda())
