"""The operators of a paged KV cache held in 8 bits, as cases that can be timed.

Four entry points are measured, in the order in which a serving step makes them:

* ``np_block_map``: block tables, slot mapping, positions and query starts of a
  batch from its requests' lengths, blocks taken from and given back to a free
  list, on the GPU.
* ``np_kv_append_q8``: new tokens' K and V quantised into pools of e4m3 or int8
  with one power-of-two scale per (block of tokens, kv head).
* ``np_paged_decode_q8``: the decode read of such a cache (one or several query
  tokens a row).
* ``np_paged_prefill_q8``: attention of ragged chunks over such a cache.

The scale of a block and head is the least power of two 2^e, e in [-60, 60], with
max |x| <= QMAX 2^e over what the block holds (QMAX: 448 for e4m3, 127 for int8).
A call that writes a block's first slot starts the block anew; one that adds to a
block keeps the larger of the old scale and the new tokens' own, and what the block
held is rounded again where the scale grew.

``run`` computes them in their plain form from elementary torch operations in
fp32, or through the library where ``own`` is true.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ cases --
def _maps(name, **kw):
    c = dict(op="maps", name=name, rows=64, singles=64, new_lo=1, new_hi=1, ctx_lo=16, ctx_hi=16384,
             block_size=16, pad=0, lens=1)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(op="append", name=name, rows=64, singles=64, new_lo=1, new_hi=1, ctx_lo=16, ctx_hi=16384,
             kv_heads=8, head_dim=128, dtype="bf16", form="e4m3", block_size=16, fused=False, lens=1)
    c.update(kw)
    return c


def _decode(name, **kw):
    c = dict(op="decode", name=name, rows=64, ctx_lo=1024, ctx_hi=8192, spread="even", query_len=1,
             q_heads=32, kv_heads=8, head_dim=128, dtype="bf16", form="e4m3", block_size=16, lens=1)
    c.update(kw)
    return c


def _chunk(name, **kw):
    c = dict(op="chunk", name=name, rows=1, singles=0, new_lo=16, new_hi=16, ctx_lo=1000, ctx_hi=1000,
             q_heads=32, kv_heads=8, head_dim=128, dtype="bf16", form="e4m3", block_size=16, lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # a decode step's batch: one token a row, some rows into a new block; then it is taken back
        _maps("maps decode 256", rows=256, singles=256, lens=11),
        # a scheduler's step of prompts and decoding rows, padded to a captured graph's token count
        _maps("maps prompts 64 rows", rows=64, singles=40, new_lo=200, new_hi=1100, ctx_lo=0, ctx_hi=4096,
              block_size=32, pad=1000, lens=12),
        # a decode step's batch: one token a row at the end of a started block (latency)
        _append("append decode 64", lens=21),
        # a long prompt's tokens in one call, several layers' worth of bandwidth
        _append("append prompt 16384", rows=1, singles=0, new_lo=16384, new_hi=16384, ctx_lo=0, ctx_hi=0,
                block_size=32, lens=22),
        # an fp32 model's chunks that begin inside a block, odd lengths, from the fused projection's rows
        _append("append int8 f32 chunks", rows=9, singles=2, new_lo=100, new_hi=700, ctx_lo=3, ctx_hi=2000,
                dtype="f32", form="int8", block_size=24, fused=True, lens=23),
        # an fp32 model's decode step over short histories (latency)
        _decode("decode f32 8 rows", rows=8, ctx_lo=512, ctx_hi=2048, dtype="f32", lens=31),
        # an ordinary decode batch
        _decode("decode 64 rows", lens=32),
        # long histories (bandwidth)
        _decode("decode long 16 rows", rows=16, ctx_lo=32768, ctx_hi=131072, q_heads=64, block_size=32,
                lens=33),
        # verification of drafted tokens: four query tokens a row, int8
        _decode("decode int8 4 tokens", query_len=4, form="int8", lens=34),
        # the last 16 tokens of a prompt whose beginning is cached (latency)
        _chunk("chunk 16 of 1000", lens=41),
        # a scheduler's mixed step: 62 rows decode, two rows fill 512 tokens each
        _chunk("mixed 62+2x512", rows=64, singles=62, new_lo=512, new_hi=512, ctx_lo=1024, ctx_hi=8192,
               lens=42),
        # a chunk of a long document, most of it cached already (the largest), int8
        _chunk("chunk 1024 of 65536", new_lo=1024, new_hi=1024, ctx_lo=65536, ctx_hi=65536, q_heads=64,
               form="int8", block_size=32, lens=43),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["maps", "append", "append", "decode", "decode", "decode", "chunk", "chunk"])
        bs = rng.choice([1, 5, 8, 16, 16, 24, 32, 64])
        kv = rng.choice([1, 2, 3, 4, 8, 8, 16])
        d = rng.choice([16, 32, 64, 128, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        form = rng.choice(["e4m3", "int8"])
        lens = rng.randrange(1 << 20)
        rows = _log(rng, 1, 1024)
        singles = rng.choice([0, rows // 2, rows])
        new_hi = _log(rng, 1, 4096)
        new_lo = rng.choice([1, new_hi])
        ctx_hi = rng.choice([0, _log(rng, 16, 32768)])
        ctx_lo = rng.choice([0, ctx_hi // 4, ctx_hi])
        if op == "maps":
            c = _maps(None, rows=rows, singles=singles, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo,
                      ctx_hi=ctx_hi, block_size=bs, pad=rng.choice([0, 0, _log(rng, 1, 512)]), lens=lens)
        elif op == "append":
            c = _append(None, rows=rows, singles=singles, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo,
                        ctx_hi=ctx_hi, kv_heads=kv, head_dim=d, dtype=dtype, form=form, block_size=bs,
                        fused=rng.random() < 0.5, lens=lens)
        elif op == "decode":
            group = rng.choice([1, 2, 3, 4, 5, 8] + ([16] if dtype == "bf16" else []))
            hi = _log(rng, 1, 65536)
            c = _decode(None, rows=_log(rng, 1, 256), ctx_lo=rng.choice([1, hi // 8 + 1, hi]), ctx_hi=hi,
                        spread=rng.choice(["even", "log"]),
                        query_len=rng.choice([1, 1, max(1, (16 if dtype == "bf16" else 8) // group // 2)]),
                        q_heads=kv * group, kv_heads=kv, head_dim=d, dtype=dtype, form=form, block_size=bs,
                        lens=lens)
        else:
            group = rng.choice([1, 2, 3, 4, 5, 8] + ([16] if dtype == "bf16" else []))
            rows = _log(rng, 1, 64)
            c = _chunk(None, rows=rows, singles=rng.choice([0, 0, rows // 2]), new_lo=new_lo,
                       new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, q_heads=kv * group, kv_heads=kv,
                       head_dim=d, dtype=dtype, form=form, block_size=bs, lens=lens)
        del c["name"]
        new, ctx = _lengths(c)
        if sum(new) > 16384 or sum(ctx) > 1 << 20:
            continue
        w, top = work(c), {x["name"]: work(x) for x in listed()}
        if op == "maps" and sum(ctx) * c["rows"] > 1 << 28:
            continue
        if op == "append" and w["bytes"] > top["append prompt 16384"]["bytes"]:
            continue
        if op == "decode" and w["bytes"] > top["decode long 16 rows"]["bytes"]:
            continue
        if op == "chunk" and w["flops"] > top["chunk 1024 of 65536"]["flops"] * (0.1 if dtype == "f32" else 0.5):
            continue
        return c


def _lengths(c):
    """(new tokens, context including them) of every row: plain lists, set by the case alone.
    ctx_lo..ctx_hi is the range of what the cache holds already ("maps", "append") or of the whole
    context ("decode", "chunk": a row whose draw is under its new tokens has no more than those)."""
    r = random.Random(c["lens"])
    new, ctx = [], []
    for i in range(c["rows"]):
        if c["op"] == "decode":
            lo, hi = c["ctx_lo"], c["ctx_hi"]
            x = r.randint(lo, hi) if c["spread"] == "even" else int(round(lo * (hi / lo) ** r.random()))
            new.append(c["query_len"])
            ctx.append(max(x, c["query_len"]))
            continue
        n = 1 if i < c["singles"] else r.randint(c["new_lo"], c["new_hi"])
        x = r.randint(c["ctx_lo"], c["ctx_hi"])
        new.append(n)
        ctx.append(max(n, x) if c["op"] == "chunk" else x + n)
    order = list(range(c["rows"]))
    r.shuffle(order)  # single-token rows stand among the others
    return [new[i] for i in order], [ctx[i] for i in order]


def work(case):
    new, ctx = _lengths(case)
    bs, rows, tokens = case["block_size"], case["rows"], sum(new)
    if case["op"] == "maps":
        # a step and its undoing: lengths read and written, slots and positions written, the taken
        # blocks' table entries and list entries both ways
        taken = sum(-(-c // bs) - -(-(c - n) // bs) for n, c in zip(new, ctx))
        return {"bytes": 2 * (16 * rows + 4 * (rows + 1)) + 12 * (tokens + case["pad"]) + 16 * taken + 16,
                "flops": 10 * (tokens + rows)}
    hk, d, es = case["kv_heads"], case["head_dim"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        touched = sum(-(-c // bs) - (c - n) // bs for n, c in zip(new, ctx))
        # K and V read, their 8-bit values written, the touched blocks' scales written, slots
        return {"bytes": 2 * tokens * hk * d * (es + 1) + 8 * touched * hk + 8 * tokens,
                "flops": 2 * tokens * hk * d * 3}
    blocks = sum(-(-c // bs) for c in ctx)
    hq = case["q_heads"]
    pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, ctx))  # (token, visible position)
    return {"bytes": 2 * tokens * hq * d * es + 2 * sum(ctx) * hk * d + blocks * (8 * hk + 4) + 8 * rows,
            "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------------- inputs --
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _form(case):
    return torch.float8_e4m3fn if case["form"] == "e4m3" else torch.int8


def _pow2(e):
    """2^e in fp32 of whole numbers e in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _need(amax, form):
    """The least e in [-60, 60] with amax <= QMAX 2^e."""
    m, ex = torch.frexp(amax)
    top, at = (0.875, 9) if form == "e4m3" else (0.9921875, 7)  # QMAX = top 2^at
    return torch.where(amax == 0, -60, ex - at + (m > top).int()).clamp(-60, 60)


def _code(y, form):
    """Scaled fp32 values to their 8-bit codes: nearest, ties to even."""
    q = QMAX[form]
    if form == "e4m3":
        return y.clamp(-q, q).to(torch.float8_e4m3fn)
    return y.round().clamp(-q, q).to(torch.int8)


def _values(gen, shape):
    """Keys or values [..., heads, dim]: heads and tokens of different sizes."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return x * torch.exp(0.4 * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))


def _pool(gen, shape, form):
    """A pool [blocks, block size, heads, dim] of 8-bit codes and its scales [blocks, heads]."""
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn if form == "e4m3" else torch.int8, device="cuda")
    scale = torch.empty((shape[0], shape[2]), device="cuda")
    step = max(1, (1 << 28) // (shape[1] * shape[2] * shape[3]))
    for b in range(0, shape[0], step):
        x = _values(gen, (min(step, shape[0] - b),) + shape[1:])
        e = _need(x.abs().amax((1, 3)), form)
        codes[b:b + step] = _code(x * _pow2(-e)[:, None, :, None], form)
        scale[b:b + step] = _pow2(e)
    return codes, scale


def _tables(need, spare, cpu, width):
    """Block tables of rows that hold need[r] blocks, and the list of the blocks that are left."""
    nb = sum(need) + spare
    ids = torch.randperm(nb, generator=cpu).to(torch.int32)
    n = torch.tensor(need)
    j = torch.arange(width)
    at = (n.cumsum(0) - n)[:, None] + j
    tables = torch.where(j < n[:, None], ids[at.clamp(max=nb - 1)], -1)
    return tables.to(torch.int32), ids[sum(need):], nb


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1))
    cpu = torch.Generator().manual_seed(7919 * (seed + 1))
    make = {"maps": _prepare_maps, "append": _prepare_append, "decode": _prepare_read, "chunk": _prepare_read}
    return make[case["op"]](case, gen, cpu)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_maps(case, gen, cpu):
    new, ctx = _lengths(case)
    bs, tokens = case["block_size"], sum(new) + case["pad"]
    have = [-(-(c - n) // bs) for n, c in zip(new, ctx)]
    width = max(-(-c // bs) for c in ctx) + 4
    taken = sum(-(-c // bs) for c in ctx) - sum(have)
    tables, left, nb = _tables(have, taken + 100, cpu, width)
    free = torch.full((nb,), -1, dtype=torch.int32)
    free[:len(left)] = left
    old = _i32([c - n for n, c in zip(new, ctx)])
    rows = case["rows"]
    return dict(case=case, tables=tables.cuda(), context_lens=old, kept=old.clone(), new=_i32(new),
                none=torch.zeros_like(old), free=free.cuda(), count=_i32([len(left)]),
                starts=torch.zeros(rows + 1, dtype=torch.int32, device="cuda"),
                starts_after=torch.zeros(rows + 1, dtype=torch.int32, device="cuda"),
                slots=torch.zeros(tokens, dtype=torch.int64, device="cuda"),
                positions=torch.zeros(tokens, dtype=torch.int32, device="cuda"))


def _prepare_append(case, gen, cpu):
    new, ctx = _lengths(case)
    bs, hk, d, dt = case["block_size"], case["kv_heads"], case["head_dim"], _dtype(case)
    # the pool: the blocks that the call touches, and some that it does not
    first = [(c - n) // bs for n, c in zip(new, ctx)]
    need = [-(-c // bs) - f for c, f in zip(ctx, first)]
    tables, _, nb = _tables(need, 8, cpu, max(need))
    n, c, f = (torch.tensor(x) for x in (new, ctx, first))
    row = torch.repeat_interleave(torch.arange(len(new)), n)
    pos = torch.arange(sum(new)) - (n.cumsum(0) - n)[row] + (c - n)[row]
    slots = tables[row, pos // bs - f[row]].long() * bs + pos % bs
    t = len(row)
    if case["fused"]:  # views of the fused projection's rows: four query heads a kv head before them
        rows = _values(gen, (t, 6 * hk, d)).to(dt)
        k, v = rows[:, 4 * hk:5 * hk], rows[:, 5 * hk:]
    else:
        k, v = (_values(gen, (t, hk, d)).to(dt) for _ in range(2))
    k_pool, k_scale = _pool(gen, (nb, bs, hk, d), case["form"])
    v_pool, v_scale = _pool(gen, (nb, bs, hk, d), case["form"])
    return dict(case=case, k=k, v=v, slots=slots.cuda(), k_pool=k_pool, v_pool=v_pool, k_scale=k_scale,
                v_scale=v_scale)


def _prepare_read(case, gen, cpu):
    new, ctx = _lengths(case)
    hq, hk, d, bs, dt = case["q_heads"], case["kv_heads"], case["head_dim"], case["block_size"], _dtype(case)
    need = [-(-c // bs) for c in ctx]
    tables, _, nb = _tables(need, 16, cpu, max(need))
    k_pool, k_scale = _pool(gen, (nb, bs, hk, d), case["form"])
    v_pool, v_scale = _pool(gen, (nb, bs, hk, d), case["form"])
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    q = torch.randn((starts[-1], hq, d), generator=gen, device="cuda").to(dt)
    groups = {}
    for r, n in enumerate(new):  # rows with equally many new tokens: one padded batch of the plain form
        groups.setdefault(n, []).append(r)
    s = dict(case=case, k_pool=k_pool, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale, tables=tables.cuda(),
             context_lens=_i32(ctx), query_starts=_i32(starts), scale=1.0 / math.sqrt(d),
             groups=[(n, torch.tensor(rows, device="cuda"), max(ctx[r] for r in rows))
                     for n, rows in groups.items()],
             # the library's workspaces: their documented size that covers every shape
             workspace=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))
    if case["op"] == "decode" and case["query_len"] > 1:
        q = q.view(case["rows"], case["query_len"], hq, d)
    s["q"], s["out"] = q, torch.zeros_like(q)
    return s


# -------------------------------------------------------------- one pass --
def run(state):
    op = state["case"]["op"]
    if own:
        return {"maps": _own_maps, "append": _own_append, "decode": _own_decode, "chunk": _own_chunk}[op](state)
    return {"maps": _run_maps, "append": _run_append, "decode": _run_read, "chunk": _run_read}[op](state)


def _maps_out(s):
    return {k: s[k] for k in ("slots", "positions", "starts", "tables", "context_lens", "free", "count")}


def _append_out(s):
    return {k: s[k] for k in ("k_pool", "v_pool", "k_scale", "v_scale")}


def _own_maps(s):
    import paged_kv_decode_np_gb300 as npg
    bs = s["case"]["block_size"]
    npg.np_block_map(s["tables"], s["context_lens"], s["new"], s["free"], s["count"], s["starts"], s["slots"],
                     s["positions"], bs, kept_lens=s["kept"])
    # the step is taken back: its blocks return to the list
    npg.np_block_map(s["tables"], s["context_lens"], s["none"], s["free"], s["count"], s["starts_after"], None,
                     None, bs, kept_lens=s["kept"])
    return _maps_out(s)


def _own_append(s):
    import paged_kv_decode_np_gb300 as npg
    npg.np_kv_append_q8(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["k"], s["v"], s["slots"])
    return _append_out(s)


def _own_decode(s):
    import paged_kv_decode_np_gb300 as npg
    npg.np_paged_decode_q8(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["tables"],
                           s["context_lens"], s["scale"], s["workspace"])
    return s["out"]


def _own_chunk(s):
    import paged_kv_decode_np_gb300 as npg
    npg.np_paged_prefill_q8(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["tables"],
                            s["context_lens"], s["query_starts"], s["scale"], s["workspace"])
    return s["out"]


def _map_step(s, new, starts, slots, positions):
    """One step of np_block_map: rows keep min(context, kept) positions and get new[r] more.  Blocks
    that are no longer needed go to the free list's end, the last row's last block first; blocks that
    are needed come from its end, for the first row's first one first."""
    bs, tables = s["case"]["block_size"], s["tables"]
    c0 = s["context_lens"]
    base = torch.minimum(c0, s["kept"])
    c1 = base + new
    have, need = (c0 + bs - 1) // bs, (c1 + bs - 1) // bs
    j = torch.arange(tables.shape[1], device="cuda")
    back = (j >= need[:, None]) & (j < have[:, None])
    take = (j >= have[:, None]) & (j < need[:, None])
    n = s["free"].numel()
    rank = back.flatten().cumsum(0) - 1
    freed = (have - need).clamp(min=0).sum()
    at = torch.where(back.flatten(), s["count"] + freed - 1 - rank, n)
    ids = torch.cat([s["free"], s["free"][:1]]).scatter(0, at.long(), tables.flatten())[:n]
    count = s["count"] + freed
    rank = take.flatten().cumsum(0) - 1
    got = ids[(count - 1 - rank).clamp(0, n - 1).long()].view_as(tables)
    tables.copy_(torch.where(take, got, torch.where(back, -1, tables)))
    s["free"].copy_(ids)
    s["count"].copy_(count - (need - have).clamp(min=0).sum())
    c0.copy_(c1)
    starts[1:] = new.cumsum(0)
    if slots is not None:
        i = torch.arange(slots.numel(), device="cuda")
        row = torch.searchsorted(starts[1:], i, right=True, out_int32=True).clamp(max=len(new) - 1).long()
        pos = base[row] + i - starts[row]
        live = i < starts[-1]
        pos = torch.where(live, pos, 0)
        block = tables[row, pos // bs].long()
        slots.copy_(torch.where(live, block * bs + pos % bs, -1))
        positions.copy_(pos)


def _run_maps(s):
    _map_step(s, s["new"], s["starts"], s["slots"], s["positions"])
    _map_step(s, s["none"], s["starts_after"], None, None)
    return _maps_out(s)


def _run_append(s):
    _append_one(s, s["k"], s["k_pool"], s["k_scale"])
    _append_one(s, s["v"], s["v_pool"], s["v_scale"])
    return _append_out(s)


def _append_one(s, x, pool, scale):
    form, (nb, bs, hk, d) = s["case"]["form"], pool.shape
    x, block = x.float(), s["slots"] // bs
    amax = torch.zeros((nb, hk), device="cuda").scatter_reduce_(0, block[:, None].expand(-1, hk),
                                                                x.abs().amax(2), "amax")
    touched = torch.zeros(nb, dtype=torch.int32, device="cuda").index_fill_(0, block, 1)
    anew = torch.zeros(nb, dtype=torch.int32, device="cuda")
    anew.index_add_(0, block, (s["slots"] % bs == 0).int())
    e = _need(amax, form)
    e_old = torch.frexp(scale)[1] - 1
    kept = torch.where(touched[:, None] > 0, torch.maximum(e_old, e), e_old)
    grew = torch.where(anew[:, None] > 0, 0, e_old - kept)
    e = torch.where(anew[:, None] > 0, e, kept)
    # what the blocks held, rounded again (by 2^0 where the scale is the old one)
    pool.copy_(_code(pool.float() * _pow2(grew.clamp(min=-126))[:, None, :, None], form))
    scale.copy_(_pow2(e))
    pool.view(-1, hk, d)[s["slots"]] = _code(x * _pow2(-e[block])[..., None], form)


def _run_read(s):
    q = s["q"].flatten(0, -3)
    out = s["out"].view_as(q)
    for n, rows, most in s["groups"]:
        _rows_read(s, s["case"], q, out, n, rows, most)
    return s["out"]


def _rows_read(s, c, q, out, n, rows, most):
    """The rows (an index tensor) with n new tokens each, contexts up to ``most``."""
    hq, hk, d, bs = c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    g = hq // hk
    ctx = s["context_lens"][rows].long()[:, None]  # [R, 1]
    tok = s["query_starts"][rows].long()[:, None] + torch.arange(n, device="cuda")  # [R, n]
    at = torch.arange(most, device="cuda")
    block = s["tables"][rows].long().clamp(min=0)[:, at // bs]  # [R, C]
    slots = block * bs + at % bs
    q = q[tok].view(len(rows), n, hk, g, d)
    sees = at <= (ctx - n + torch.arange(n, device="cuda"))[..., None]  # [R, n, C]
    live = (at < ctx)[..., None, None]
    # as many kv heads at a time as keep the scores and the widened values under 2^31 elements
    step = max(1, min(hk, (1 << 31) // (len(rows) * most * max(g * n, d))))
    for h in range(0, hk, step):
        e = min(hk, h + step)
        k = s["k_pool"].view(-1, hk, d)[slots, h:e].float() * s["k_scale"][block, h:e][..., None]
        v = s["v_pool"].view(-1, hk, d)[slots, h:e].float() * s["v_scale"][block, h:e][..., None]
        v = torch.where(live, v, 0.0).transpose(1, 2)
        x = q[:, :, h:e].float().permute(0, 2, 1, 3, 4).reshape(len(rows), e - h, n * g, d)
        x = torch.matmul(x, k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(len(rows), e - h, n, g, most)
        x.masked_fill_(~sees[:, None, :, None], -math.inf)
        x = x.sub_(x.amax(-1, keepdim=True)).exp_()  # every token sees itself at least
        z = x.sum(-1, keepdim=True)
        y = torch.matmul(x.view(len(rows), e - h, n * g, most), v).view(len(rows), e - h, n, g, d) / z
        out.view(-1, hk, g, d)[:, h:e][tok] = y.transpose(1, 2).to(_dtype(c))


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The operators' definitions in 64 bits, on prepare()'s inputs."""
    if case["op"] in ("decode", "chunk") and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "maps":
        return _exact_maps(case, s)
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_read(case, s)


def _exact_maps(case, s):
    """Request by request on the host."""
    bs, (new, ctx) = case["block_size"], _lengths(case)
    tables, free = s["tables"].tolist(), s["free"].tolist()
    top = int(s["count"])
    slots, positions, starts, taken = [], [], [0], []
    for r, (n, c) in enumerate(zip(new, ctx)):
        for j in range(-(-(c - n) // bs), -(-c // bs)):
            top -= 1
            tables[r][j] = free[top]
            taken.append((r, j))
        for t in range(c - n, c):
            slots.append(tables[r][t // bs] * bs + t % bs)
            positions.append(t)
        starts.append(len(slots))
    while taken:  # undone: the last one taken goes back first
        r, j = taken.pop()
        free[top], tables[r][j] = tables[r][j], -1
        top += 1
    slots += [-1] * case["pad"]
    positions += [0] * case["pad"]
    return {"slots": torch.tensor(slots), "positions": _i32(positions), "starts": _i32(starts),
            "tables": _i32(tables), "context_lens": _i32([c - n for n, c in zip(new, ctx)]),
            "free": _i32(free), "count": _i32([top])}


def _two(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(y, form):
    """The nearest representable value of 64-bit y, ties to even, no further than QMAX."""
    if form == "int8":
        return y.round().clamp(-127, 127)
    size = y.abs().clamp(min=2.0 ** -40).log2().floor()
    size = size + (y.abs() >= _two(size + 1)).double() - (y.abs() < _two(size)).double()
    grain = _two(size.clamp(min=-6) - 3)  # three bits after the leading one; from 2^-9 on below 2^-6
    return (y / grain).round().mul(grain).clamp(-448, 448)


def _exact_append(case, s):
    form, bs = case["form"], case["block_size"]
    out = {}
    for name in "kv":
        pool, scale = s[name + "_pool"].double(), s[name + "_scale"].double()
        x, slots = s[name].double(), s["slots"]
        powers = _two(torch.arange(-60, 61, device="cuda"))
        need = torch.full_like(scale, 2.0 ** -60)
        amax = torch.zeros_like(scale)
        index = (slots // bs)[:, None].expand(-1, scale.shape[1])
        amax.scatter_reduce_(0, index, x.abs().amax(-1), "amax")
        need = powers[torch.searchsorted(powers * QMAX[form], amax).clamp(max=120)]
        written = torch.zeros(pool.shape[0] * bs, dtype=torch.bool, device="cuda")
        written[slots] = True
        written = written.view(-1, bs)
        anew, some = written[:, :1], written.any(1, keepdim=True)
        after = torch.where(anew, need, torch.where(some, torch.maximum(scale, need), scale))
        factor = torch.where(anew, 1.0, scale / after)
        pool = torch.where(factor[:, None, :, None] == 1, pool, _nearest(pool * factor[:, None, :, None], form))
        pool.flatten(0, 1)[slots] = _nearest(x / after[slots // bs][..., None], form)
        out[name + "_pool"] = pool if form == "e4m3" else pool.to(torch.int8)
        out[name + "_scale"] = after
    return out


def _exact_read(case, s):
    new, ctx = _lengths(case)
    g, d, bs = case["q_heads"] // case["kv_heads"], case["head_dim"], case["block_size"]
    q = s["q"].reshape(-1, case["q_heads"], d)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    first = 0
    for r, (n, c) in enumerate(zip(new, ctx)):
        blocks = s["tables"][r, :-(-c // bs)].long()
        ahead = torch.ones(n, c, dtype=torch.bool, device="cuda").triu(c - n + 1)
        for h in range(case["kv_heads"]):
            k, v = ((s[p + "_pool"][blocks, :, h].double() * s[p + "_scale"][blocks, h].double()[:, None, None])
                    .reshape(-1, d)[:c] for p in "kv")
            qh = q[first:first + n, h * g:h * g + g].double().transpose(0, 1)  # [g, n, d]
            z = (qh @ k.T) * s["scale"]
            z.masked_fill_(ahead, -math.inf)
            out[first:first + n, h * g:h * g + g] = \
                (torch.exp(z - torch.logsumexp(z, -1, keepdim=True)) @ v).transpose(0, 1)
        first += n
    return out.view(s["q"].shape)
