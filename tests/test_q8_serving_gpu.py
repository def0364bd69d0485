"""The 8-bit cache's calls together, as a serving loop makes them."""
import pytest
import torch

import q8_helpers as h
from prompt_helpers import chunk_reference, chunk_tolerance

pytestmark = pytest.mark.gpu


class Server:
    """Requests whose K and V are known in full: every output is compared with attention over what
    the cache's own codes stand for, and the codes with the values they were made from."""

    def __init__(self, npg, form, dtype, rows=5, bs=16, hk=2, g=4, d=64, mb=24, nb=60):
        self.npg, self.form, self.dtype, self.bs, self.hk, self.g, self.d = npg, form, dtype, bs, hk, g, d
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cache = npg.q8_pools(nb, bs, hk, d, form)
        self.tables, self.lens = torch.full((rows, mb), -1, **i32), torch.zeros(rows, **i32)
        self.free, self.count = torch.randperm(nb).to("cuda", torch.int32), torch.tensor([nb], **i32)
        self.starts, self.err = torch.zeros(rows + 1, **i32), torch.zeros(1, **i32)
        self.slots = torch.zeros(400, dtype=torch.int64, device="cuda")
        self.positions = torch.zeros(400, **i32)
        self.new, self.kept = torch.zeros(rows, **i32), torch.zeros(rows, **i32)
        self.q = torch.zeros(400, hk * g, d, dtype=dtype, device="cuda")
        self.k, self.v = (torch.zeros(400, hk, d, dtype=dtype, device="cuda") for _ in range(2))
        self.out = torch.zeros_like(self.q)
        self.ws = npg.prefill_workspace(d)
        self.wd = npg.decode_q8_workspace(d)
        self.true = [[torch.zeros(0, hk, d) for _ in range(2)] for _ in range(rows)]
        self.seed = 0

    def launch(self):
        """Bookkeeping, append, attention: nothing of it waits for the host."""
        npg = self.npg
        npg.np_block_map(self.tables, self.lens, self.new, self.free, self.count, self.starts, self.slots,
                         self.positions, self.bs, kept_lens=self.kept, err_word=self.err)
        npg.prefill_step_q8(self.out, self.q, self.k, self.v, self.slots, *self.cache, self.tables, self.lens,
                            self.starts, 0.1, self.ws, err_word=self.err)

    def step(self, new, kept, run):
        gen = torch.Generator().manual_seed(self.seed)
        self.seed += 1
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=gen))
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.kept.copy_(torch.tensor(kept, dtype=torch.int32))
        at = 0
        for r, n in enumerate(new):
            for i, t in enumerate((self.k, self.v)):
                self.true[r][i] = torch.cat([self.true[r][i][:kept[r]], t[at:at + n].float().cpu()])
            at += n
        self.out.fill_(77.0)
        run()
        torch.cuda.synchronize()
        assert int(self.err) == 0
        ctx = [len(t[0]) for t in self.true]
        assert self.lens.tolist() == ctx
        rows = list(zip(new, ctx))
        inp = dict(q=self.q, k_pool=h.widened(self.cache[0], self.cache[2]),
                   v_pool=h.widened(self.cache[1], self.cache[3]), block_tables=self.tables,
                   context_lens=self.lens, query_starts=self.starts)
        ref, bound = chunk_reference(inp, rows, 0.1)
        tol = chunk_tolerance(ref, bound, self.dtype, self.d, max(ctx + [1]))
        used = sum(new)
        assert ((self.out[:used].double() - ref[:used]).abs() <= tol[:used]).all()
        assert (self.out[used:] == 77.0).all()
        # the codes: at most the last rounding's half step and as much from those before it
        for r, c in enumerate(ctx):
            t = torch.arange(c, device="cuda")
            b = self.tables[r].long()[t // self.bs]
            for i in range(2):
                s = self.cache[2 + i][b][..., None].cpu().double()
                got = self.cache[i][b, t % self.bs].float().cpu().double() * s
                true = self.true[r][i].double()
                step = s if self.form is torch.int8 else torch.maximum(true.abs() / 8, s * 2.0 ** -9)
                assert ((got - true).abs() <= step).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", list(h.FORMS.values()), ids=list(h.FORMS))
def test_prompts_decode_drafts_and_release(nplib, form, dtype):
    s = Server(nplib, form, dtype)
    s.step([100, 17, 1, 0, 40], [0] * 5, s.launch)          # prompts
    s.step([60, 1, 30, 5, 1], [100, 17, 1, 0, 40], s.launch)  # chunks among decoding rows
    s.step([4] * 5, [160, 18, 31, 5, 41], s.launch)          # drafted tokens
    s.step([4] * 5, [161, 22, 33, 6, 44], s.launch)          # some of them rejected
    s.step([0, 4, 50, 1, 90], [0, 26, 0, 10, 48], s.launch)  # one request ends, another takes a row over
    s.step([120, 1, 1, 1, 1], [0, 30, 50, 11, 138], s.launch)


def test_a_captured_step_replayed(nplib):
    """The whole step in one graph: bookkeeping, append and attention, sizes from the device."""
    s = Server(nplib, torch.float8_e4m3fn, torch.bfloat16)
    s.step([30, 1, 2, 3, 4], [0] * 5, s.launch)
    saved = [t.clone() for t in (s.tables, s.lens, s.free, s.count, *[c.view(torch.uint8) for c in s.cache])]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.launch()
    # (capturing runs nothing)
    for t, x in zip((s.tables, s.lens, s.free, s.count, *[c.view(torch.uint8) for c in s.cache]), saved):
        assert torch.equal(t, x)
    s.step([1, 100, 1, 1, 33], [30, 1, 2, 3, 4], g.replay)
    s.step([1, 1, 1, 200, 1], [31, 101, 0, 4, 30], g.replay)
    s.step([0, 0, 0, 0, 0], [32, 102, 1, 204, 31], g.replay)


@pytest.mark.parametrize("form", list(h.FORMS.values()), ids=list(h.FORMS))
def test_the_decode_read_after_a_prompt(nplib, form):
    """decode_step_q8 on the same cache: one and several tokens a row."""
    s = Server(nplib, form, torch.bfloat16)
    s.step([100, 17, 1, 9, 40], [0] * 5, s.launch)
    for ql in (1, 4):
        rows = 5

        def run(ql=ql):
            nplib.np_block_map(s.tables, s.lens, s.new, s.free, s.count, s.starts, s.slots[:rows * ql],
                               s.positions[:rows * ql], s.bs, kept_lens=s.kept, err_word=s.err)
            view = (rows, ql, -1, s.d) if ql > 1 else (rows, -1, s.d)
            nplib.decode_step_q8(s.out[:rows * ql].view(view), s.q[:rows * ql].view(view), *s.cache, s.tables,
                                 s.lens, 0.1, s.wd, k_new=s.k[:rows * ql].view(view),
                                 v_new=s.v[:rows * ql].view(view), slot_mapping=s.slots[:rows * ql].view(rows, ql),
                                 err_word=s.err)

        s.step([ql] * rows, s.lens.tolist(), run)


def test_rotated_keys_into_the_cache(nplib):
    """np_rope_append rotates into a staging pool of one block, np_kv_append_q8 rounds from there."""
    npg, t, hk, hq, d = nplib, 70, 2, 8, 64
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(t, n, d, generator=gen).to("cuda", torch.bfloat16) for n in (hq, hk, hk))
    table = npg.rope_table(256, d)
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    stage_k, stage_v = (torch.zeros(1, t, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qr = torch.empty_like(q)
    npg.np_rope_append(qr, q, k, v, pos.long(), stage_k, stage_v, table, pos)
    cache = npg.q8_pools(6, 16, hk, d)
    slots = pos.long() + 16
    npg.np_kv_append_q8(*cache, stage_k[0], stage_v[0], slots)
    half = d // 2
    c, s = table[:t, None, :half].double(), table[:t, None, half:].double()
    x = k.double()
    turned = torch.cat([x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s], -1)
    got = h.widened(cache[0], cache[2]).flatten(0, 1)[slots]
    scale = cache[2][slots // 16].double()[..., None]
    # bf16's half step, then e4m3's
    assert ((got - turned).abs() <= turned.abs() * (2.0 ** -8 + 2.0 ** -4 * 1.01) + scale * 2.0 ** -10 + 1e-6).all()


def test_two_reads_at_once(nplib):
    """Two streams, each with its own workspace and output, on one cache."""
    rows = [(1, c) for c in (3000, 50, 700)]
    inp = h.read_inputs(torch.bfloat16, torch.int8, 128, 8, 4, 16, rows)
    args = [inp[k] for k in ("k_pool", "v_pool", "k_scale", "v_scale", "block_tables", "context_lens")]

    def read(out, ws):
        nplib.np_paged_decode_q8(out, inp["q"], *args, 0.1, ws)

    def attend(out, ws):
        nplib.np_paged_prefill_q8(out, inp["q"], *args, inp["query_starts"], 0.1, ws)

    outs = [torch.zeros_like(inp["q"]) for _ in range(4)]
    wss = [nplib.decode_q8_workspace(128), nplib.decode_q8_workspace(128), nplib.prefill_workspace(128)]
    read(outs[3], wss[0])
    want = outs[3].clone()
    attend(outs[3], wss[2])
    want2 = outs[3].clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, fn in enumerate((read, read, attend)):
            with torch.cuda.stream(streams[i]):
                fn(outs[i], wss[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and torch.equal(outs[2], want2)


def test_tensors_off_the_current_device_are_refused(nplib):
    inp = h.read_inputs(torch.bfloat16, torch.int8, 64, 2, 2, 16, [(1, 20)])
    ws, out = nplib.decode_q8_workspace(64), torch.zeros_like(inp["q"])
    for name in ("k_pool", "v_scale", "context_lens"):
        bad = dict(inp, **{name: inp[name].cpu()})
        with pytest.raises(ValueError, match="CUDA"):
            nplib.np_paged_decode_q8(out, bad["q"], bad["k_pool"], bad["v_pool"], bad["k_scale"], bad["v_scale"],
                                     bad["block_tables"], bad["context_lens"], 0.1, ws)
    with pytest.raises(ValueError, match="contiguous"):
        nplib.np_paged_decode_q8(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["k_scale"].T.contiguous().T,
                                 inp["v_scale"], inp["block_tables"], inp["context_lens"], 0.1, ws)


def test_a_refused_step_has_written_nothing(nplib):
    """What the read or the attention refuses (too small a workspace, too many heads a kv head) is
    refused before the append; scales may begin on any four bytes."""
    npg = nplib
    i32 = dict(dtype=torch.int32, device="cuda")
    kp, vp, _, _ = npg.q8_pools(3, 16, 1, 64)
    layers = torch.zeros(2, 3, 1, device="cuda")  # a layer's scales: 12 bytes apart
    cache = (kp, vp, layers[1], torch.zeros(3, 1, device="cuda"))
    before = [t.view(torch.uint8).clone() if t.dtype is not torch.float32 else t.clone() for t in cache]
    k = torch.randn(2, 1, 64, device="cuda", dtype=torch.bfloat16)
    slots = torch.tensor([0, 16], device="cuda")
    tables, lens = torch.tensor([[0], [1]], **i32), torch.ones(2, **i32)
    starts = torch.tensor([0, 1, 2], **i32)
    small = torch.empty(1024, dtype=torch.uint8, device="cuda")
    for heads, ws in ((4, small), (17, npg.decode_q8_workspace(64))):
        q = torch.randn(2, heads, 64, device="cuda", dtype=torch.bfloat16)
        with pytest.raises(npg.NPError):
            npg.decode_step_q8(torch.empty_like(q), q, *cache, tables, lens, 0.1, ws, k_new=k, v_new=k,
                               slot_mapping=slots)
        with pytest.raises(npg.NPError):
            npg.prefill_step_q8(torch.empty_like(q), q, k, k, slots, *cache, tables, lens, starts, 0.1,
                                small if ws is small else npg.prefill_workspace(64))
    torch.cuda.synchronize()
    for t, x in zip(cache, before):
        assert torch.equal(t.view(torch.uint8) if t.dtype is not torch.float32 else t, x)
    q = torch.randn(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    out = torch.empty_like(q)
    npg.decode_step_q8(out, q, *cache, tables, lens, 0.1, npg.decode_q8_workspace(64), k_new=k, v_new=k,
                       slot_mapping=slots)
    # one position a row: its own value, by e4m3's half step, then bf16's
    assert ((out.double() - k.double()).abs() <= k.double().abs() * (2.0 ** -4 + 2.0 ** -8) * 1.01 + 2.0 ** -16).all()
    assert (layers[0] == 0).all() and (layers[1, :2] > 0).all() and (layers[1, 2] == 0).all()
