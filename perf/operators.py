"""The prompt-side operators of a paged KV cache, as cases that can be timed.

Two entry points are measured:

* ``np_rope_append``: new tokens' q, k and v; q and k are (optionally) RMS
  normalised per head and rotated by their positions, q goes to a buffer of
  its own, k and v to the tokens' slots of the paged pools, in one pass.
* ``np_paged_prefill``: attention of ragged chunks of new tokens over the
  rows' paged histories (the chunk's own tokens included, causally).

``run`` computes them in their plain form from elementary torch operations in
fp32, or through the library where ``own`` is true.
"""
import math
import random

import torch

own = False

# Rows of the rotation tables (positions a table covers).
TABLE = 131072


# ------------------------------------------------------------------ cases --
def _rope(name, **kw):
    c = dict(op="rope", name=name, tokens=64, q_heads=32, kv_heads=8, head_dim=128, rot_dim=128,
             dtype="bf16", block_size=16, kind="decode", axes=1, interleaved=False, norm=False,
             fused=False)
    c.update(kw)
    return c


def _chunk(name, **kw):
    c = dict(op="chunk", name=name, rows=1, singles=0, new_lo=16, new_hi=16, ctx_lo=1000,
             ctx_hi=1000, q_heads=32, kv_heads=8, head_dim=128, dtype="bf16", block_size=16,
             lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # a decode step's batch: one token a row, far and near positions (latency)
        _rope("rope decode 64"),
        # a long prompt's tokens in one call (bandwidth)
        _rope("rope prompt 16384", tokens=16384, q_heads=64, block_size=32, kind="prompt"),
        # a decode batch of a model that normalises q and k, from the fused projection's rows
        _rope("norm rope decode 256", tokens=256, q_heads=40, block_size=8, norm=True, fused=True),
        # an fp32 model's prompt with the norms, an odd number of tokens
        _rope("norm rope prompt f32", tokens=4099, dtype="f32", kind="prompt", norm=True),
        # image tokens of a vision-language prompt: positions in time, height and width
        _rope("rope three axes", tokens=5329, kind="image", axes=3, fused=True),
        # a small multi-axis batch of interleaved pairs with norms, narrow heads, partial rotation
        _rope("rope axes interleaved", tokens=301, q_heads=16, kv_heads=2, head_dim=64, rot_dim=32,
              dtype="f32", kind="image", axes=3, interleaved=True, norm=True),
        # the last 16 tokens of a prompt whose beginning is cached (latency)
        _chunk("chunk 16 of 1000"),
        # a scheduler's mixed step: 62 rows decode, two rows fill 512 tokens each
        _chunk("mixed 62+2x512", rows=64, singles=62, new_lo=512, new_hi=512, ctx_lo=1024,
               ctx_hi=8192, lens=2),
        # a chunk of a long document, most of it cached already (the largest)
        _chunk("chunk 1024 of 131072", new_lo=1024, new_hi=1024, ctx_lo=131072, ctx_hi=131072,
               q_heads=64, block_size=32, lens=3),
        # whole prompts of several lengths, nothing cached: causal from the first token
        _chunk("prompts 6 ragged", rows=6, new_lo=500, new_hi=4096, ctx_lo=0, ctx_hi=0, q_heads=40,
               block_size=8, lens=4),
        # an fp32 model's chunks over short histories
        _chunk("chunks f32", rows=8, new_lo=64, new_hi=192, ctx_lo=512, ctx_hi=2048, dtype="f32",
               lens=5),
        # wide heads, one kv head for eight query heads, odd chunk lengths
        _chunk("chunks wide one kv", rows=16, new_lo=17, new_hi=301, ctx_lo=640, ctx_hi=4096,
               q_heads=8, kv_heads=1, head_dim=256, lens=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        if rng.random() < 0.5:
            d = rng.choice([16, 32, 64, 128, 128, 256])
            kind = rng.choice(["decode", "prompt", "image"])
            kv = rng.choice([1, 2, 3, 4, 8, 8, 16])
            c = _rope(None, tokens=_log(rng, 1, 512) if kind == "decode" else _log(rng, 1, 16384),
                      q_heads=kv * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=kv, head_dim=d,
                      rot_dim=rng.choice([d, d, max(16, d // 2)]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                      block_size=rng.choice([1, 5, 8, 16, 32, 64]), kind=kind,
                      axes=3 if kind == "image" else 1, interleaved=rng.random() < 0.4,
                      norm=rng.random() < 0.5, fused=rng.random() < 0.5)
            del c["name"]
            if work(c)["bytes"] <= work(listed()[1])["bytes"]:
                return c
        else:
            dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
            kv = rng.choice([1, 2, 3, 4, 8, 8])
            rows = _log(rng, 1, 64)
            new_hi = _log(rng, 1, 4096)
            ctx_hi = rng.choice([0, _log(rng, 16, 65536)])
            c = _chunk(None, rows=rows, singles=rng.choice([0, 0, rows // 2]),
                       new_lo=rng.choice([1, max(1, new_hi // 2), new_hi]), new_hi=new_hi,
                       ctx_lo=rng.choice([0, ctx_hi // 4, ctx_hi]), ctx_hi=ctx_hi,
                       q_heads=kv * rng.choice([1, 2, 3, 4, 5, 8] + ([16] if dtype == "bf16" else [])),
                       kv_heads=kv, head_dim=rng.choice([32, 64, 128, 128, 256]), dtype=dtype,
                       block_size=rng.choice([1, 5, 8, 16, 16, 24, 32, 64]), lens=rng.randrange(1 << 20))
            del c["name"]
            new, ctx = _lengths(c)
            if sum(new) > 16384 or sum(ctx) > 1 << 19:
                continue
            # fp32 products take no tensor core: a tenth of the largest listed case's operations
            most = work(listed()[8])["flops"] * (0.1 if dtype == "f32" else 0.5)
            if work(c)["flops"] <= most:
                return c


def _lengths(c):
    """(new tokens, context including them) of every row: plain lists, set by the case alone.
    ctx_lo..ctx_hi is the context's range; a row whose draw is under its chunk has no more than
    the chunk (a prompt from its first token)."""
    r = random.Random(c["lens"])
    new, ctx = [], []
    for i in range(c["rows"]):
        n = 1 if i < c["singles"] else r.randint(c["new_lo"], c["new_hi"])
        new.append(n)
        ctx.append(max(n, r.randint(c["ctx_lo"], c["ctx_hi"])))
    order = list(range(c["rows"]))
    r.shuffle(order)  # single-token rows stand among the others
    return [new[i] for i in order], [ctx[i] for i in order]


def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        t = case["tokens"]
        elems = t * (hq + 2 * hk) * d
        # every input and output once: q, k, v; the rotation's table rows; positions, slots
        return {"bytes": 2 * elems * es + t * (case["rot_dim"] * 4 + 4 * case["axes"] + 8),
                "flops": t * (hq + hk) * (3 * case["rot_dim"] + (4 * d if case["norm"] else 0))}
    new, ctx = _lengths(case)
    pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, ctx))  # (token, visible position)
    tab = sum(-(-c // case["block_size"]) for c in ctx)
    return {"bytes": 2 * sum(new) * hq * d * es + 2 * sum(ctx) * hk * d * es + 4 * tab + 8 * len(new) + 4,
            "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------------- inputs --
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1))
    cpu = torch.Generator().manual_seed(7919 * (seed + 1))
    return _prepare_rope(case, gen, cpu) if case["op"] == "rope" else _prepare_chunk(case, gen, cpu)


def _sections(case):
    """Pairs of each axis: a quarter of the pairs for time, the rest halved between height and
    width."""
    half = case["rot_dim"] // 2
    if case["axes"] == 1:
        return [half]
    t = half // 4
    h = (half - t) // 2
    return [t, h, half - t - h]


def _prepare_rope(case, gen, cpu):
    t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    dt, bs = _dtype(case), case["block_size"]
    if case["fused"]:  # views of the fused projection's rows
        rows = _randn(gen, (t, (hq + 2 * hk) * d), dt)
        q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split([hq * d, hk * d, hk * d], 1))
    else:
        q, k, v = (_randn(gen, (t, h, d), dt) for h in (hq, hk, hk))
    # the rotation's angles, formed in 64 bits: a table row per position
    half = case["rot_dim"] // 2
    freq = 500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(TABLE, device="cuda", dtype=torch.float64)[:, None] * freq
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    i = torch.arange(t)
    if case["kind"] == "decode":  # every token at the end of a row of its own
        pos = torch.randint(0, TABLE, (t,), generator=cpu)[None]
        blocks = torch.randperm(t + 8, generator=cpu)[:t]
        slots = blocks * bs + torch.randint(0, bs, (t,), generator=cpu)
        nb = t + 8
    else:
        nb = -(-t // bs) + 8
        slots = torch.randperm(nb, generator=cpu)[i // bs] * bs + i % bs
        start = int(torch.randint(0, TABLE - t, (1,), generator=cpu))
        if case["kind"] == "prompt":
            pos = (start + i)[None]
        else:  # an image: one step in time, a square grid in height and width
            side = math.isqrt(max(t - 1, 0)) + 1
            pos = torch.stack([torch.full((t,), start), start + i // side, start + i % side])
    w = [1 + 0.1 * _randn(gen, (d,), torch.float32) for _ in range(2)] if case["norm"] else [None, None]
    return dict(case=case, q=q, k=k, v=v, table=table, sections=_sections(case),
                positions=(pos if case["axes"] > 1 else pos[0]).to("cuda", torch.int32).contiguous(),
                slots=slots.to("cuda", torch.int64), q_out=torch.empty((t, hq, d), dtype=dt, device="cuda"),
                k_pool=_randn(gen, (nb, bs, hk, d), dt), v_pool=_randn(gen, (nb, bs, hk, d), dt),
                q_weight=None if w[0] is None else w[0].to(dt),
                k_weight=None if w[1] is None else w[1].to(dt), eps=1e-6)


def _prepare_chunk(case, gen, cpu):
    new, ctx = _lengths(case)
    hq, hk, d, bs, dt = case["q_heads"], case["kv_heads"], case["head_dim"], case["block_size"], _dtype(case)
    need = [-(-c // bs) for c in ctx]
    nb = sum(need) + 16
    ids = torch.randperm(nb, generator=cpu).to(torch.int32)
    tables = torch.full((len(new), max(need)), -1, dtype=torch.int32)
    at = 0
    for r, m in enumerate(need):
        tables[r, :m] = ids[at:at + m]
        at += m
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    q = _randn(gen, (starts[-1], hq, d), dt)
    groups = {}
    for r, n in enumerate(new):  # rows with equally many new tokens: one padded batch of the plain form
        groups.setdefault(n, []).append(r)
    groups = [(n, torch.tensor(rows, device="cuda"), max(ctx[r] for r in rows))
              for n, rows in groups.items()]
    return dict(case=case, groups=groups, q=q, out=torch.zeros_like(q),
                k_pool=_randn(gen, (nb, bs, hk, d), dt), v_pool=_randn(gen, (nb, bs, hk, d), dt),
                tables=tables.cuda(), context_lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                query_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                scale=1.0 / math.sqrt(d),
                # the library's workspace: its documented size that covers every shape
                workspace=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))


# -------------------------------------------------------------- one pass --
def run(state):
    if state["case"]["op"] == "rope":
        return _run_rope_own(state) if own else _run_rope(state)
    return _run_chunk_own(state) if own else _run_chunk(state)


def _run_rope_own(s):
    import paged_kv_decode_np_gb300 as npg
    c = s["case"]
    npg.np_rope_append(s["q_out"], s["q"], s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"],
                       s["table"], s["positions"], sections=s["sections"] if c["axes"] > 1 else None,
                       interleaved=c["interleaved"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                       eps=s["eps"])
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _run_chunk_own(s):
    import paged_kv_decode_np_gb300 as npg
    npg.np_paged_prefill(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["context_lens"],
                         s["query_starts"], s["scale"], s["workspace"])
    return s["out"]


def _rotate(x, weight, s, cos, sin):
    """[tokens, heads, dim] -> the same, normalised (where there is a weight) and rotated, fp32."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()
    rot = c["rot_dim"]
    half = rot // 2
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return y if rot == x.shape[-1] else torch.cat([y, x[..., rot:]], -1)


def _run_rope(s):
    c = s["case"]
    half = c["rot_dim"] // 2
    if c["axes"] == 1:
        cs = s["table"][s["positions"]]
        cos, sin = cs[:, None, :half], cs[:, None, half:]
    else:  # each axis' run of pairs from that axis' table rows
        cs = s["table"][s["positions"]]  # [axes, tokens, rot]
        t, h, w = s["sections"]
        cos, sin = (torch.cat([cs[0, :, o:o + t], cs[1, :, o + t:o + t + h], cs[2, :, o + t + h:o + half]],
                              1)[:, None] for o in (0, half))
    s["q_out"].copy_(_rotate(s["q"], s["q_weight"], s, cos, sin))
    hk, d = c["kv_heads"], c["head_dim"]
    s["k_pool"].view(-1, hk, d)[s["slots"]] = _rotate(s["k"], s["k_weight"], s, cos, sin).to(_dtype(c))
    s["v_pool"].view(-1, hk, d)[s["slots"]] = s["v"]
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _run_chunk(s):
    for n, rows, most in s["groups"]:
        _rows_chunk(s, s["case"], n, rows, most)
    return s["out"]


def _rows_chunk(s, c, n, rows, most):
    """The rows (an index tensor) with n new tokens each, contexts up to ``most``."""
    hq, hk, d, bs = c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    g = hq // hk
    ctx = s["context_lens"][rows].long()[:, None]  # [R, 1]
    tok = s["query_starts"][rows].long()[:, None] + torch.arange(n, device="cuda")  # [R, n]
    at = torch.arange(most, device="cuda")
    slots = s["tables"][rows].long().clamp(min=0)[:, at // bs] * bs + at % bs  # [R, C]
    q = s["q"][tok].view(len(rows), n, hk, g, d)
    sees = at <= (ctx - n + torch.arange(n, device="cuda"))[..., None]  # [R, n, C]
    live = (at < ctx)[..., None, None]
    # as many kv heads at a time as keep the scores under 2^31 elements
    step = max(1, min(hk, (1 << 31) // (len(rows) * g * n * most)))
    for h in range(0, hk, step):
        e = min(hk, h + step)
        k = s["k_pool"].view(-1, hk, d)[slots, h:e].float().permute(0, 2, 3, 1)  # [R, H, D, C]
        v = torch.where(live, s["v_pool"].view(-1, hk, d)[slots, h:e].float(), 0.0).transpose(1, 2)
        x = q[:, :, h:e].float().permute(0, 2, 1, 3, 4).reshape(len(rows), e - h, n * g, d)
        x = torch.matmul(x, k).mul_(s["scale"]).view(len(rows), e - h, n, g, most)
        x.masked_fill_(~sees[:, None, :, None], -math.inf)
        x = x.sub_(x.amax(-1, keepdim=True)).exp_()  # every token sees itself at least
        z = x.sum(-1, keepdim=True)
        y = torch.matmul(x.view(len(rows), e - h, n * g, most), v).view(len(rows), e - h, n, g, d) / z
        s["out"].view(-1, hk, g, d)[:, h:e][tok] = y.transpose(1, 2).to(_dtype(c))


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The operators' definitions in 64 bits, on prepare()'s inputs."""
    if case["op"] == "chunk" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    new, ctx = _lengths(case)
    g, d = case["q_heads"] // case["kv_heads"], case["head_dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for r, (n, c) in enumerate(zip(new, ctx)):
        blocks = s["tables"][r, :-(-c // case["block_size"])].long()
        ahead = torch.ones(n, c, dtype=torch.bool, device="cuda").triu(c - n + 1)
        for h in range(case["kv_heads"]):
            k = s["k_pool"][blocks, :, h].reshape(-1, d)[:c].double()
            v = s["v_pool"][blocks, :, h].reshape(-1, d)[:c].double()
            for j in range(h * g, h * g + g):
                z = (s["q"][first:first + n, j].double() @ k.T) * s["scale"]
                z.masked_fill_(ahead, -math.inf)
                out[first:first + n, j] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ v
        first += n
    return out


def _exact_rope(case, s):
    """Each pair as a complex number, times cos + i sin of its axis' position."""
    half, t = case["rot_dim"] // 2, case["tokens"]
    axis = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(s["sections"])).cuda()
    where = s["positions"].view(case["axes"], t)[axis].long()  # [half, tokens]
    j = torch.arange(half, device="cuda")[:, None]
    turn = torch.complex(s["table"][where, j].double(), s["table"][where, j + half].double()).T[:, None]

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * weight.double()
        x = x.clone()
        even, odd = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else \
            (slice(0, half), slice(half, 2 * half))
        y = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * turn
        x[..., even], x[..., odd] = y.real, y.imag
        return x

    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    k_pool.flatten(0, 1)[s["slots"]] = turned(s["k"], s["k_weight"])
    v_pool.flatten(0, 1)[s["slots"]] = s["v"].double()
    return {"q": turned(s["q"], s["q_weight"]), "k_pool": k_pool, "v_pool": v_pool}
