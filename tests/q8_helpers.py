"""Plain 64-bit implementations of the 8-bit cache's operators, for the tests."""
from __future__ import annotations

import math

import torch

from prompt_helpers import HALF, chunk_tolerance

FORMS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def least_exponent(amax: float, qmax: float) -> int:
    """The least e in [-60, 60] with amax <= qmax 2^e, by trying."""
    for e in range(-60, 61):
        if amax <= qmax * 2.0 ** e:
            return e
    return 60


def nearest(y: torch.Tensor, form) -> torch.Tensor:
    """The nearest code's value, ties to even, at most QMAX, of 64-bit y (CPU); NaN: NaN or 0."""
    if form is torch.int8:
        return torch.nan_to_num(y, nan=0.0, posinf=127.0, neginf=-127.0).round().clamp(-127, 127)
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 0 .. 448
    a = y.abs().clamp(max=448.0)
    hi = torch.searchsorted(codes, torch.nan_to_num(a, nan=0.0)).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - codes[lo], codes[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return torch.where(y.isnan(), y, torch.copysign(codes[pick], y))


def append_reference(pool, scale, x, slots):
    """np_kv_append_q8 of one of K and V on the host: (code values as 64 bits, exponents)."""
    form, (nb, bs, hk, d) = pool.dtype, pool.shape
    q = QMAX[form]
    val = pool.cpu().float().double()
    exp = torch.tensor([[max(-60, min(60, math.frexp(abs(s))[1] - 1)) if 0 < abs(s) < math.inf else
                         (-60 if s == 0 else 60) for s in row] for row in scale.cpu().tolist()])
    out_e = exp.clone()
    x = x.cpu().double()
    slots = slots.cpu().tolist()
    by_block = {}
    for i, s in enumerate(slots):
        if 0 <= s < nb * bs:
            by_block.setdefault(s // bs, []).append(i)
    for b, toks in by_block.items():
        offs = {slots[i] % bs: i for i in toks}
        for h in range(hk):
            v = x[toks, h]
            fin = v[v.isfinite()]
            e = least_exponent(float(fin.abs().max()) if fin.numel() else 0.0, q)
            if 0 not in offs:
                e = max(e, int(exp[b, h]))
                if e > int(exp[b, h]):
                    for o in range(bs):
                        if o not in offs:
                            val[b, o, h] = nearest(val[b, o, h] * 2.0 ** (int(exp[b, h]) - e), form)
            for o, i in offs.items():
                val[b, o, h] = nearest(x[i, h] * 2.0 ** -e, form)
            out_e[b, h] = e
    touched = sorted(by_block)
    return val, out_e, touched


def random_cache(nb, bs, hk, d, form, gen, spread=2):
    """(k_pool, v_pool, k_scale, v_scale) of random codes under random scales, on the CPU."""
    def pool():
        if form is torch.int8:
            return torch.randint(-127, 128, (nb, bs, hk, d), generator=gen, dtype=torch.int16).to(torch.int8)
        return (torch.randn(nb, bs, hk, d, generator=gen) * 100).clamp(-448, 448).to(form)

    def scale():
        e = torch.randint(-spread, spread + 1, (nb, hk), generator=gen)
        return torch.ldexp(torch.ones(nb, hk), e - (7 if form is torch.int8 else 8))

    return pool(), pool(), scale(), scale()


def widened(pool, scale):
    """The 64-bit values that a cache stands for."""
    return pool.float().double() * scale.double()[:, None, :, None]


def read_inputs(dtype, form, d, hk, g, bs, rows, *, seed=0, before=0, behind=0, spare=3, cap=None,
                spread=2, dev="cuda"):
    """Inputs of the 8-bit reads.  rows: [(n, c)].  Slots that hold no history are NaN or -128,
    blocks that hold none have scales that are no powers of two, unused table entries are -1;
    `before` and `behind` tokens of q belong to no row."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-c // bs) for _, c in rows]
    nb = sum(need) + spare
    ids = torch.randperm(nb, generator=gen).to(torch.int32)
    mb = max([1] + need) if cap is None else cap
    tables = torch.full((len(rows), mb), -1, dtype=torch.int32)
    kp, vp, ks, vs = random_cache(nb, bs, hk, d, form, gen, spread)
    live = torch.zeros(nb * bs, dtype=torch.bool)
    at, starts = 0, [before]
    for r, (n, c) in enumerate(rows):
        tables[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
        t = torch.arange(c)
        live[tables[r, t // bs].long() * bs + t % bs] = True
        starts.append(starts[-1] + n)
    for p in (kp, vp):
        p.view(torch.uint8).view(nb * bs, hk, d)[~live] = 0x80 if form is torch.int8 else 0x7f
    unused = ids[sum(need):].long()
    ks[unused], vs[unused] = float("nan"), float("inf")
    tokens = starts[-1] + behind
    q = torch.randn(tokens, hk * g, d, generator=gen).to(dtype)
    t32 = dict(dtype=torch.int32, device=dev)
    return dict(q=q.to(dev), k_pool=kp.to(dev), v_pool=vp.to(dev), k_scale=ks.to(dev),
                v_scale=vs.to(dev), block_tables=tables.to(dev),
                context_lens=torch.tensor([c for _, c in rows], **t32),
                query_starts=torch.tensor(starts, **t32))


def as_values(inp):
    """The same inputs with pools of 64-bit values (for prompt_helpers.chunk_reference)."""
    return dict(inp, k_pool=widened(inp["k_pool"], inp["k_scale"]), v_pool=widened(inp["v_pool"], inp["v_scale"]))


def decode_tolerance(ref, bound, dtype, d, longest, vtop):
    """How far np_paged_decode_q8 may be off, per element.

    Scores: a sum of d products, off by at most d 2^-23 of the sum of the products' sizes (an
    accumulator may truncate), its scaling, the shift of M and V's exponent by 4 x 2^-23 of sizes no
    larger than that sum and 2^7 (an exponent of at most 60 and the shift of 14 are added in);
    fp32: q is off by 2^-22 of itself in its two parts.  The exponential of that, relative, and 2^-22
    of the function's own; twice, for numerator and denominator.  Sums over `longest` positions:
    longest 2^-23 of theirs, twice.  A weight is rounded to fp16 (half a step 2^-11), or to two parts
    (2^-22); one below fp16's normals is off by at most 2^-25 where the largest is 2^6 or more, which
    moves the result by at most 2^-31 of the largest value, each.  bf16's result is rounded once."""
    mass, big = bound
    e = (d + 4) * 2.0 ** -23 * big + 4 * 2.0 ** -23 * 128 * 0.7 + 2.0 ** -22
    if dtype == torch.float32:
        e = e + 2.0 ** -22 * big
    tol = mass * (2 * e + 2 * longest * 2.0 ** -23)
    tol = tol + mass * (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22)
    tol = tol + longest * 2.0 ** -31 * vtop
    return 1.1 * (tol + HALF[dtype] * ref.abs()) + 1e-30


def prefill_tolerance(inp, ref, bound, dtype, d, longest, scale):
    """How far np_paged_prefill_q8 may be off, per element: prompt_helpers.chunk_tolerance, and for
    bf16 with tiled copies what fp16 adds at its small end.

    A weight below fp16's normals is off by at most 2^-25 where the largest is 2^6 or more: 2^-31 of
    the largest value, for each of `longest` positions (a value of 0 under the largest weight leaves
    nothing else to compare with).  A V element whose block's scale is far below its tile's is off by at
    most 2^-25 of the tile's scale, 2^-31 of the largest value and less; weights add up to 1.  A K
    element, likewise, by 2^-25 of the tile's scale: a score by that times the sum of |q|, and the output
    by twice that, relative."""
    tol = chunk_tolerance(ref, bound, dtype, d, longest)
    bs = inp["k_pool"].shape[1]
    if dtype != torch.bfloat16 or d < 64 or bs % 8 or longest == 0:
        return tol
    used = inp["block_tables"][inp["block_tables"] >= 0].long()
    if used.numel() == 0:
        return tol
    top = {k: float(inp[k][used].clamp(2.0 ** -60, 2.0 ** 60).max()) for k in ("k_scale", "v_scale")}
    vtop = top["v_scale"] * QMAX[inp["v_pool"].dtype]
    inside = ~ref.isnan()
    q = inp["q"].double().abs().sum(-1, keepdim=True).expand(inp["q"].shape)
    if q.shape != ref.shape:  # (the caller left out tokens of no row)
        starts = inp["query_starts"].tolist()
        q = q[starts[0]:starts[-1]]
    e = q * abs(scale) * 2.0 ** -25 * top["k_scale"]
    return tol + torch.where(inside, 1.1 * (2 * e * bound[0] + (longest + 1) * 2.0 ** -31 * vtop), 0.0)
