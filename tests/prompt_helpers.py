"""Plain 64-bit implementations of the prompt-side operators, for the tests."""
from __future__ import annotations

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def chunk_inputs(dtype, d, hk, g, bs, rows, *, seed=0, before=0, behind=0, spare=3, cap=None,
                 poison=True, dev="cuda"):
    """Inputs of np_paged_prefill.  rows: [(n, c)].  Slots that hold no history are NaN, unused
    table entries -1, `before` and `behind` tokens of q belong to no row."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-c // bs) for _, c in rows]
    nb = sum(need) + spare
    ids = torch.randperm(nb, generator=gen).to(torch.int32)
    mb = max([1] + need) if cap is None else cap
    tables = torch.full((len(rows), mb), -1, dtype=torch.int32)
    k = torch.full((nb * bs, hk, d), float("nan") if poison else 0.0)
    v = k.clone()
    at, starts = 0, [before]
    for r, (n, c) in enumerate(rows):
        tables[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
        t = torch.arange(c)
        slots = tables[r, t // bs].long() * bs + t % bs
        k[slots] = torch.randn(c, hk, d, generator=gen)
        v[slots] = torch.randn(c, hk, d, generator=gen)
        starts.append(starts[-1] + n)
    tokens = starts[-1] + behind
    q = torch.randn(tokens, hk * g, d, generator=gen)
    return dict(q=q.to(dtype).to(dev), k_pool=k.view(nb, bs, hk, d).to(dtype).to(dev),
                v_pool=v.view(nb, bs, hk, d).to(dtype).to(dev), block_tables=tables.to(dev),
                context_lens=torch.tensor([c for _, c in rows], dtype=torch.int32, device=dev),
                query_starts=torch.tensor(starts, dtype=torch.int32, device=dev))


def chunk_reference(inp, rows, scale):
    """(out, bound) in 64 bits: the attention of every chunk token of every row, and the same sums
    over |v| with the largest sum of |q k| products (for the tolerance).  Tokens of no row: NaN."""
    q, kp, vp = inp["q"], inp["k_pool"], inp["v_pool"]
    bs, hk, d = kp.shape[1:]
    g = q.shape[1] // hk
    starts = inp["query_starts"].tolist()
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    mass = torch.zeros_like(out)
    big = torch.zeros(q.shape[:2] + (1,), dtype=torch.float64, device=q.device)
    for r, (n, c) in enumerate(rows):
        s = starts[r]
        nblk = -(-c // bs)
        blocks = inp["block_tables"][r, :nblk].long()
        kh = kp[blocks].reshape(nblk * bs, hk, d)[:c].double()
        vh = vp[blocks].reshape(nblk * bs, hk, d)[:c].double()
        for i in range(n):
            m = max(0, c - n + i + 1)  # positions seen
            if m == 0:
                out[s + i] = 0
                continue
            qi = q[s + i].double().view(hk, g, d)
            z = torch.einsum("hgd,thd->hgt", qi, kh[:m]) * scale
            p = torch.softmax(z, -1)
            out[s + i] = torch.einsum("hgt,thd->hgd", p, vh[:m]).reshape(hk * g, d)
            mass[s + i] = torch.einsum("hgt,thd->hgd", p, vh[:m].abs()).reshape(hk * g, d)
            zz = torch.einsum("hgd,thd->hgt", qi.abs(), kh[:m].abs()).amax(-1) * abs(scale)
            big[s + i] = zz.reshape(hk * g, 1)
    return out, (mass, big)


def chunk_tolerance(ref, bound, dtype, d, longest):
    """How far a kernel with fp32 sums may be off, per element.

    A score is a sum of d products: off by at most d 2^-23 of the sum of the products' sizes (2^-23:
    an accumulator may truncate), its scaling and the subtraction of the maximum by 4 x 2^-23 of
    sizes no larger; so its exponential is off by that, relative, plus 2^-22 of the function's own.
    A relative error e in every weight moves the output by at most 2 e of sum p |v| (numerator and
    denominator).  Sums over `longest` positions add longest 2^-23 of the same, twice.  bf16: each
    weight is rounded to bf16 for its product with v (half a step of sum p |v|), and the result
    once (half a step of itself).  Scores differ from the exact ones by less than 0.1, so second
    order terms are within a tenth: the factor 1.1."""
    mass, big = bound
    e = (d + 4) * 2.0 ** -23 * big + 2.0 ** -22
    tol = 1.1 * mass * (2 * e + 2 * longest * 2.0 ** -23)
    if dtype == torch.bfloat16:
        tol = tol + 1.1 * (HALF[dtype] * mass + HALF[dtype] * ref.abs())
    else:
        tol = tol + HALF[dtype] * ref.abs()
    return tol + 1e-30


def rope_reference(q, k, table, positions, sections, interleaved, qw, kw, eps):
    """(q, k) rotated in 64 bits, and for each the sizes |x0 c| + |x1 s| (for the tolerance)."""
    rot = table.shape[1]
    half = rot // 2
    pos = positions.view(-1, positions.shape[-1]).long().clamp(0, table.shape[0] - 1)
    sections = [half] if sections is None else list(sections)
    axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device=pos.device)
    j = torch.arange(half, device=pos.device)
    c = table[pos[axis].T, j].double()[:, None]          # [T, 1, half]
    s = table[pos[axis].T, half + j].double()[:, None]
    i0 = 2 * j if interleaved else j
    i1 = 2 * j + 1 if interleaved else j + half

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x * w.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        y, size = x.clone(), x.abs()
        x0, x1 = x[..., i0], x[..., i1]
        y[..., i0], y[..., i1] = x0 * c - x1 * s, x1 * c + x0 * s
        size[..., i0] = (x0 * c).abs() + (x1 * s).abs()
        size[..., i1] = (x1 * c).abs() + (x0 * s).abs()
        return y, size

    return one(q, qw) if q is not None else None, one(k, kw)


def rope_tolerance(y, size, dtype, d, norm):
    """Two products, a sum: 3 roundings of 2^-24 of the sizes at most.  With a norm, the sum of d
    squares is off by (d + 1) 2^-24, its root and the quotient by half of that and 2 x 2^-24 each,
    two more products: (d / 2 + 8) 2^-24.  The result is rounded to the type once."""
    e = (3 + (d / 2 + 8 if norm else 0)) * 2.0 ** -24
    return 1.01 * e * size + 1.01 * (HALF[dtype] * y.abs() if dtype == torch.bfloat16 else 0) + 1e-37
