"""np_kv_append_q8 against its definition, code by code."""
import pytest
import torch

import q8_helpers as h

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _append(npg, cache, k, v, slots):
    cache = [t.cuda() for t in cache]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    npg.np_kv_append_q8(*cache, k, v, slots.cuda(), err_word=err)
    torch.cuda.synchronize()
    return [t.cpu() for t in cache], int(err)


def _check(npg, cache, k, v, slots, flags=0):
    got, err = _append(npg, cache, k, v, slots)
    assert err == flags
    for i, x in ((0, k), (1, v)):
        val, e, touched = h.append_reference(cache[i], cache[2 + i], x, slots)
        untouched = [b for b in range(val.shape[0]) if b not in touched]
        assert torch.equal(got[i].view(torch.uint8)[untouched], cache[i].view(torch.uint8)[untouched])
        assert torch.equal(got[2 + i][untouched], cache[2 + i][untouched])
        assert torch.equal(got[2 + i][touched].double(), 2.0 ** e[touched].double())
        same = (got[i].float().double() == val) | (got[i].float().isnan() & val.isnan())
        # (a code of -128, of garbage, is rounded to -127 only where its block's scale grew)
        assert same[touched].all()


def _slots(rows, bs, gen, spare=3):
    """Slots of the new tokens of rows [(old, new)], blocks drawn from a shuffled list."""
    need = [-(-(c + n) // bs) for c, n in rows]
    nb = sum(need) + spare
    ids = torch.randperm(nb, generator=gen)
    out, at = [], 0
    for (c, n), m in zip(rows, need):
        t = torch.arange(c, c + n)
        out.append(ids[at + t // bs] * bs + t % bs)
        at += m
    return torch.cat(out), nb


@pytest.mark.parametrize("form", list(h.FORMS.values()), ids=list(h.FORMS))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("bs", [1, 5, 16, 64])
def test_rows_of_many_kinds(nplib, bs, d, dtype, form):
    gen = torch.Generator().manual_seed(d + bs)
    rows = [(0, 1), (3, 1), (0, 37), (bs - 1, 1), (bs, 2), (7, 90), (0, bs), (1, bs)]
    slots, nb = _slots(rows, bs, gen)
    cache = h.random_cache(nb, bs, 3, d, form, gen, spread=6)
    t = len(slots)
    size = torch.exp(torch.randn(t, 3, 1, generator=gen) * 2)
    k, v = ((torch.randn(t, 3, d, generator=gen) * size).to(dtype).cuda() for _ in range(2))
    _check(nplib, cache, k, v, slots)


@pytest.mark.parametrize("hk", [1, 2, 7, 16])
@pytest.mark.parametrize("t", [1, 31, 512, 600, 5000])
def test_token_counts(nplib, t, hk):
    """Each way of dealing tokens over thread blocks; runs that cross their borders."""
    gen = torch.Generator().manual_seed(t + hk)
    slots, nb = _slots([(5, t)], 24, gen)
    cache = h.random_cache(nb, 24, hk, 32, torch.float8_e4m3fn, gen)
    k, v = (torch.randn(t, hk, 32, generator=gen).to(BF16).cuda() for _ in range(2))
    _check(nplib, cache, k, v, slots)


@pytest.mark.parametrize("form", list(h.FORMS.values()), ids=list(h.FORMS))
def test_padding_and_slots_past_the_pool(nplib, form):
    gen = torch.Generator().manual_seed(1)
    bs, nb = 8, 6
    cache = h.random_cache(nb, bs, 2, 64, form, gen)
    slots = torch.tensor([-1, 3, 4, -7, 16, 17, 18, nb * bs, nb * bs + 5, 1 << 40, 40, -1])
    k, v = (torch.randn(len(slots), 2, 64, generator=gen).cuda() for _ in range(2))
    _check(nplib, cache, k, v, slots, nplib.NP_FLAG_SLOT)


@pytest.mark.parametrize("form", list(h.FORMS.values()), ids=list(h.FORMS))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_values_at_the_borders(nplib, dtype, form):
    """Largest values at a scale's end and just past it; ties; subnormal codes; zeros; sizes beyond
    both ends of the scales."""
    q = h.QMAX[form]
    bs, d = 4, 16
    eps = torch.finfo(dtype).eps
    tops = [q, q * (1 + eps), q * 2.0 ** 20, q * (1 - eps / 2), 1.0, 2.0 ** -70, 0.0, 2.0 ** 75, 1.7e38, 1e-40]
    nb = len(tops)
    gen = torch.Generator().manual_seed(2)
    cache = h.random_cache(nb, bs, 1, d, form, gen)
    cache = [*cache[:2], torch.zeros(nb, 1), torch.zeros(nb, 1)]
    k = torch.zeros(nb, 1, d)
    for i, top in enumerate(tops):
        k[i, 0, 0] = top
        k[i, 0, 1:9] = top * torch.tensor([-1, 0.5, 0.75 / q, 1.5 / q, 2.5 / q, -3.5 / q, 17.0 / 16 / 2, 2.0 ** -16])
        k[i, 0, 9] = -0.0
    k = k.to(dtype).cuda()
    for off in (0, 2):  # anew, and into a block that holds something
        _check(nplib, cache, k, k.flip(0), torch.arange(nb) * bs + off)


@pytest.mark.parametrize("form", list(h.FORMS.values()), ids=list(h.FORMS))
def test_values_that_are_not_finite(nplib, form):
    gen = torch.Generator().manual_seed(3)
    cache = h.random_cache(4, 8, 2, 32, form, gen)
    k = torch.randn(5, 2, 32, generator=gen)
    k[0, 0, 3], k[1, 1, 5], k[2, 0, 0] = float("inf"), float("-inf"), float("nan")
    k[4] = float("nan")
    _check(nplib, cache, k.cuda(), torch.randn(5, 2, 32, generator=gen).cuda(), torch.tensor([0, 1, 2, 9, 16]),
           nplib.NP_FLAG_VALUE)


def test_a_scale_that_grows_step_by_step(nplib):
    """Token by token into one block: the scale only grows, what was there is rounded again."""
    gen = torch.Generator().manual_seed(4)
    for form in h.FORMS.values():
        cache = h.random_cache(2, 16, 2, 64, form, gen)
        true = torch.zeros(16, 2, 64, dtype=torch.float64)
        for i in range(16):
            k = torch.randn(1, 2, 64, generator=gen) * 2.0 ** (i * 0.6)
            true[i] = k[0].double()
            _check(nplib, cache, k.cuda(), k.cuda(), torch.tensor([16 + i]))
            cache, _ = _append(nplib, cache, k.cuda(), k.cuda(), torch.tensor([16 + i]))
        # roundings of growing steps: the last one's half, and as much again from those before
        s = cache[2][1].double()[None, :, None]
        step = s if form is torch.int8 else torch.maximum(true.abs() / 8, s * 2.0 ** -9)
        assert ((h.widened(cache[0], cache[2])[1] - true).abs() <= step).all()


def test_strided_tokens(nplib):
    """Views of a fused projection's rows."""
    gen = torch.Generator().manual_seed(6)
    for dtype in (BF16, F32):
        rows = torch.randn(100, 12, 64, generator=gen).to(dtype).cuda()
        cache = h.random_cache(9, 16, 2, 64, torch.float8_e4m3fn, gen)
        _check(nplib, cache, rows[:, 8:10], rows[:, 10:], torch.arange(100) + 16)


def test_stored_scales_of_any_bits(nplib):
    """A scale that is found counts as its exponent, clamped."""
    gen = torch.Generator().manual_seed(7)
    wild = torch.tensor([[0.0], [5.9], [-0.3], [float("inf")], [1e-38], [3e38], [2.0 ** -60]])
    cache = [*h.random_cache(7, 4, 1, 16, torch.int8, gen)[:2], wild.clone(), wild.flip(0).clone()]
    k = torch.randn(7, 1, 16, generator=gen).cuda()
    _check(nplib, cache, k, k, torch.arange(7) * 4 + 2)
