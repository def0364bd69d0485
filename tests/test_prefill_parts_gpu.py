"""np_paged_prefill on fp32 pools: every product of parts that a score is made of arrives in it.

The kernel takes an fp32 number as three bf16 ones (8 significant bits each) and adds six of the nine
products.  Here the large products cancel, two dims against one another, and what is left of a score is
one product of two named parts, the same for half of the positions and zero for the others: were it lost
or overwritten, all scores of a row would be equal and the halves' weights too."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

W = 127  # seven bits


def _operands(a, b):
    """q, K without and K with the product of q's part a and K's part b: two dims each.  A number's
    parts are its first 8 significant bits, the next 8 of the rest, and what remains:
    1 | W 2^-14, or 1 | 2^-9 | W 2^-23."""
    fine, x = W * 2.0 ** -14, 1 + 2.0 ** -9
    return {(0, 0): ((1.0, 0.0), (0.0, 0.0), (1.0, 0.0)),
            (0, 1): ((1.0, -1.0), (1.0, 1.0), (1 + fine, 1.0)),
            (1, 0): ((1 + fine, -1.0), (0.0, 0.0), (1.0, 1.0)),
            (1, 1): ((1 + fine, -1.0), (1.0, 1 + fine), (1 + fine, 1 + 2 * fine)),
            (0, 2): ((1.0, -1.0), (x, x), (x + W * 2.0 ** -23, x)),
            (2, 0): ((x + W * 2.0 ** -23, -x), (0.0, 0.0), (1.0, 1.0))}[a, b]


def _parts(x):
    out, x = [], torch.tensor(x, dtype=torch.float32)
    for _ in range(3):
        y = (x.view(torch.int32) & -65536).view(torch.float32)
        out.append(y.double())
        x = x - y
    assert (x == 0).all()
    return out


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("a,b", [(0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0)])
@pytest.mark.parametrize("negative", [False, True])
def test_every_product_of_parts_reaches_the_score(nplib, d, a, b, negative):
    c, n, g, bs, at = 200, 3, 2, 16, d - 2  # four kv tiles; the two dims are the last ones
    q2, off, on = (torch.tensor(z, dtype=torch.float64) for z in _operands(a, b))
    size = float(q2 @ on)
    assert float(q2 @ off) == 0 and size == float(_parts(q2.tolist())[a] @ (
        torch.stack(_parts(on.tolist()))[b] - torch.stack(_parts(off.tolist()))[b])) \
        if (a, b) != (1, 1) else size == (W * 2.0 ** -14) ** 2
    gen = torch.Generator().manual_seed(d + 10 * a + b)
    has = torch.randint(0, 2, (c,), generator=gen).bool()
    nb = -(-c // bs) + 1
    k, v = torch.zeros(2, nb * bs, 1, d, dtype=torch.float64)
    k[:c, 0, at:] = torch.where(has[:, None], on, off)
    v[:c][has] = 1.0  # an output is the weight of the positions that have the product
    q = torch.zeros(n, g, d, dtype=torch.float64)
    q[..., at:] = q2
    assert torch.equal(k, k.float().double()) and torch.equal(q, q.float().double())
    scale = 3.5 / size * (-1 if negative else 1)
    out = torch.zeros(n, g, d, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    nplib.np_paged_prefill(out, q.float().cuda(), k.float().view(nb, bs, 1, d).cuda(),
                           v.float().view(nb, bs, 1, d).cuda(),
                           torch.arange(nb, dtype=torch.int32, device="cuda")[None],
                           torch.tensor([c], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale,
                           nplib.prefill_workspace(d), err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    # A step of the matrix unit adds up to three numbers here that are not zero (two products and
    # what it has so far), none above 2; each may be cut at 2^-23 of the largest.  Six such steps a
    # score: it is off by less than 2 x 18 x 2^-23, the difference of two scores by twice that, and
    # the ratio of the halves' weights by the exponential of that times the scale.  A hundredth more
    # for all roundings of 2^-15 and below (exponentials, sums, the result).
    slack = 4 * 18 * 2.0 ** -23 * abs(scale)
    assert slack < 3.0  # less than the 3.5 that would be lost
    for i in range(n):
        m = c - n + i + 1
        ones = int(has[:m].sum())
        base = math.log(ones / (m - ones))
        got = out[i].cpu().double()
        odds = torch.log(got / (1 - got))
        want = base + (-3.5 if negative else 3.5)
        assert ((odds - want).abs() <= slack + 0.01).all(), (odds - want, slack)
