"""The prompt-side calls' refusals, on the CPU: every call here fails validation or has nothing to do
before anything touches a device."""
import ctypes

import pytest
import torch

FAKE = 0x100000  # an aligned address that is never dereferenced
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from paged_kv_decode_np_gb300 import build_lib
    path = build_lib.build()
    import paged_kv_decode_np_gb300 as npg
    return npg.load(path)


def _rope(lib, **kw):
    # addresses far enough apart for the sizes below
    a = dict(qo=FAKE, q=FAKE + MB, k=FAKE + 2 * MB, v=FAKE + 3 * MB, qs=512, ks=256, vs=256, sm=FAKE,
             kp=FAKE + 4 * MB, vp=FAKE + 5 * MB, dtype=1, nb=16, bs=16, hq=4, hk=2, d=128, cs=FAKE,
             mp=100, rot=128, pos=FAKE, axes=1, sec=None, inter=0, qw=None, kw=None, eps=1e-6, n=3,
             err=None)
    a.update(kw)
    sec = None if a["sec"] is None else (ctypes.c_int32 * len(a["sec"]))(*a["sec"])
    return lib.np_rope_append(a["qo"], a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["sm"],
                              a["kp"], a["vp"], a["dtype"], a["nb"], a["bs"], a["hq"], a["hk"], a["d"],
                              a["cs"], a["mp"], a["rot"], a["pos"], a["axes"], sec, a["inter"], a["qw"],
                              a["kw"], a["eps"], a["n"], a["err"], None)


def test_rope_append_refusals(lib):
    assert _rope(lib, n=0) == 0
    assert _rope(lib, n=-1) == 1
    assert _rope(lib, dtype=3) == 2
    assert _rope(lib, d=80, rot=80) == 2
    assert _rope(lib, rot=24) == 2                     # not a multiple of 16
    assert _rope(lib, rot=144) == 1                    # more than the head
    assert _rope(lib, rot=0) == 1
    assert _rope(lib, axes=5, sec=[64, 0, 0, 0, 0]) == 2
    assert _rope(lib, axes=0) == 1
    assert _rope(lib, axes=3) == 1                     # several axes need sections
    assert _rope(lib, axes=3, sec=[16, 24, 23]) == 1   # do not add up
    assert _rope(lib, axes=2, sec=[-1, 65]) == 1
    assert _rope(lib, axes=2, sec=[2**31 - 1, 2**31 - 1]) == 1
    assert _rope(lib, eps=-1.0) == 1
    assert _rope(lib, eps=float("nan")) == 1
    assert _rope(lib, eps=float("inf")) == 1
    assert _rope(lib, inter=2) == 1
    assert _rope(lib, mp=0) == 1
    assert _rope(lib, hq=-1) == 1
    assert _rope(lib, hk=0) == 1
    assert _rope(lib, hk=5000) == 2
    assert _rope(lib, nb=2**62) == 4
    assert _rope(lib, qs=2**61, n=100) == 4            # token offsets past 64 bits
    assert _rope(lib, qs=511) == 1                     # tokens run into one another
    assert _rope(lib, qs=516) == 1                     # not a multiple of 16 bytes
    assert _rope(lib, ks=255) == 1
    assert _rope(lib, vs=260) == 1
    for name in ("k", "v", "sm", "kp", "vp", "cs", "pos", "q", "qo"):
        assert _rope(lib, **{name: None}) == 1, name
        if name not in ("sm", "pos"):
            assert _rope(lib, **{name: FAKE + 7 * MB + 8}) == 1, name
    assert _rope(lib, sm=FAKE + 4) == 1
    assert _rope(lib, pos=FAKE + 2) == 1
    assert _rope(lib, err=FAKE + 2) == 1
    assert _rope(lib, qw=FAKE + 8) == 1
    assert _rope(lib, kw=FAKE + 8) == 1
    # no q heads: q and q_out must be absent, and the other way round
    assert _rope(lib, hq=0) == 1
    assert _rope(lib, hq=0, q=None, qo=None, qw=FAKE) == 1
    # what is written overlaps what is read
    assert _rope(lib, qo=FAKE + MB + 1024) == 1
    assert _rope(lib, qo=FAKE + MB, qs=1024) == 1      # in place, but q is strided
    assert _rope(lib, kp=FAKE + MB) == 1
    assert _rope(lib, vp=FAKE + 2 * MB) == 1
    assert _rope(lib, kp=FAKE) == 1
    assert _rope(lib, kp=FAKE + 5 * MB + 16) == 1      # the pools overlap


def test_rope_append_accepts(lib):
    # without a GPU the launch itself fails with NP_ERR_CUDA
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    assert _rope(lib) == 5
    assert _rope(lib, qo=FAKE + MB) == 5               # in place
    assert _rope(lib, qo=FAKE + MB, qs=4096, n=1) == 5
    assert _rope(lib, hq=0, q=None, qo=None) == 5
    assert _rope(lib, axes=3, sec=[16, 24, 24]) == 5
    assert _rope(lib, hq=5) == 1                       # (q tokens 512 elements apart overlap)
    assert _rope(lib, hq=3, kw=FAKE, eps=0.0) == 5


def _prefill(lib, **kw):
    a = dict(out=FAKE, q=FAKE + MB, k=FAKE + 2 * MB, v=FAKE + 3 * MB, dtype=1, nb=16, bs=16, hk=2, d=128,
             bt=FAKE, mb=4, cl=FAKE, qs=FAKE, rows=2, n=5, hq=4, scale=0.1, ws=FAKE + 8 * MB,
             wsb=1 << 30, err=None)
    a.update(kw)
    return lib.np_paged_prefill(a["out"], a["q"], a["k"], a["v"], a["dtype"], a["nb"], a["bs"], a["hk"],
                                a["d"], a["bt"], a["mb"], a["cl"], a["qs"], a["rows"], a["n"], a["hq"],
                                a["scale"], a["ws"], a["wsb"], a["err"], None)


def test_prefill_refusals(lib):
    assert _prefill(lib, rows=0) == 0
    assert _prefill(lib, n=0) == 0
    assert _prefill(lib, rows=-1) == 1
    assert _prefill(lib, n=-1) == 1
    assert _prefill(lib, dtype=2) == 2
    assert _prefill(lib, d=48) == 2
    assert _prefill(lib, hq=3) == 1
    assert _prefill(lib, hk=1, hq=17) == 2
    assert _prefill(lib, hk=1, hq=9, dtype=0) == 2
    assert _prefill(lib, scale=float("nan")) == 1
    assert _prefill(lib, scale=float("inf")) == 1
    assert _prefill(lib, bs=0) == 1
    assert _prefill(lib, mb=0) == 1
    assert _prefill(lib, rows=4097) == 2
    assert _prefill(lib, mb=2**20, bs=2**12) == 2      # positions past int32
    assert _prefill(lib, n=2**31 - 1) == 2
    assert _prefill(lib, nb=2**62) == 4
    for name in ("out", "q", "k", "v", "bt", "cl", "qs"):
        assert _prefill(lib, **{name: None}) == 1, name
    for name in ("out", "q", "k", "v"):
        assert _prefill(lib, **{name: FAKE + 7 * MB + 8}) == 1, name
    for name in ("bt", "cl", "qs", "err"):
        assert _prefill(lib, **{name: FAKE + 2}) == 1, name
    assert _prefill(lib, out=FAKE + MB) == 1           # out overlaps q
    assert _prefill(lib, out=FAKE + MB + 512) == 1
    assert _prefill(lib, out=FAKE + 2 * MB) == 1       # out overlaps a pool
    assert _prefill(lib, ws=None) == 3
    assert _prefill(lib, wsb=1000) == 3
    assert _prefill(lib, ws=FAKE + 8 * MB + 128) == 3


def test_packed_calls_check_the_same(lib):
    assert lib.np_rope_append_packed(None) == 1
    assert lib.np_paged_prefill_packed(None) == 1
    import paged_kv_decode_np_gb300 as npg
    # rows 0: nothing to do; a q_heads that kv_heads does not divide: refused
    form = npg._PREFILL_ARGS
    args = [FAKE, FAKE + MB, FAKE + 2 * MB, FAKE + 3 * MB, FAKE, FAKE, FAKE, FAKE + 8 * MB, 0, 0, 16,
            1 << 30, 1, 16, 2, 128, 4, 0, 5, 4, 0.1]
    assert lib.np_paged_prefill_packed(form.pack(*args)) == 0
    args[-2] = 3
    assert lib.np_paged_prefill_packed(form.pack(*args)) == 1
    args[-2], args[17], args[11] = 4, 2, -5
    assert lib.np_paged_prefill_packed(form.pack(*args)) == 3  # a negative workspace size
    form = npg._ROPE_ARGS
    args = [FAKE, FAKE + MB, FAKE + 2 * MB, FAKE + 3 * MB, FAKE, FAKE + 4 * MB, FAKE + 5 * MB, FAKE, FAKE,
            0, 0, 0, 0, 512, 256, 256, 16, 1, 16, 4, 2, 128, 100, 128, 3, 0, 0, 1, 16, 24, 24, 0, 1e-6]
    assert lib.np_rope_append_packed(form.pack(*args)) == 0    # no tokens
    args[29] = 23
    assert lib.np_rope_append_packed(form.pack(*args)) == 1    # sections do not add up
    args[29], args[24] = 24, 5
    assert lib.np_rope_append_packed(form.pack(*args)) == 2    # five axes


def test_prefill_workspace(lib):
    import paged_kv_decode_np_gb300 as npg
    f = lib.np_paged_prefill_workspace_bytes
    assert f(100) == 0 and f(0) == 0 and f(-16) == 0
    for d in (16, 32, 64, 128, 256):
        assert 0 < f(d) <= npg.NP_PREFILL_WORKSPACE_BYTES
    with pytest.raises(ValueError):
        npg.prefill_workspace(48, device="cpu")


def test_binding_refusals():
    import paged_kv_decode_np_gb300 as npg
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    pool, slots = torch.zeros(4, 16, 2, 64), torch.zeros(3, dtype=torch.int64)
    tab, pos = torch.zeros(9, 64), torch.zeros(3, dtype=torch.int32)

    def rope(**kw):
        a = dict(q_out=q.clone(), q=q, k_new=k, v_new=k, slot_mapping=slots, k_pool=pool, v_pool=pool,
                 cos_sin=tab, positions=pos)
        a.update(kw)
        return npg.np_rope_append(**a)

    for kw, what in [(dict(), "CUDA"), (dict(k_new=k[:2]), "k_new/v_new"),
                     (dict(v_pool=pool.bfloat16()), "dtype"), (dict(q=None), "go together"),
                     (dict(q=q[:2]), "q must be"), (dict(q_out=q[:2]), "q_out must match"),
                     (dict(q=q.bfloat16()), "q must be"), (dict(slot_mapping=slots.int()), "slot_mapping"),
                     (dict(cos_sin=tab.double()), "cos_sin"), (dict(positions=pos.long()), "positions"),
                     (dict(positions=pos[:2]), "positions"), (dict(sections=(16, 16)), "section"),
                     (dict(q_weight=torch.ones(32)), "q_weight"),
                     (dict(k_weight=torch.ones(64).bfloat16()), "k_weight")]:
        with pytest.raises(ValueError, match=what):
            rope(**kw)
    bt, cl = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    qs = torch.zeros(3, dtype=torch.int32)

    def prefill(**kw):
        a = dict(out=q.clone(), q=q, k_pool=pool, v_pool=pool, block_tables=bt, context_lens=cl,
                 query_starts=qs, scale=0.1, workspace=None)
        a.update(kw)
        return npg.np_paged_prefill(**a)

    for kw, what in [(dict(), "CUDA"), (dict(q=q[0]), "q must be"), (dict(out=q[:2]), "out must match"),
                     (dict(v_pool=pool[:2]), "mismatch"), (dict(q=q.bfloat16()), "mismatch"),
                     (dict(block_tables=bt.long()), "block_tables"), (dict(context_lens=cl[:1]), "context"),
                     (dict(query_starts=qs[:2]), "query_starts"), (dict(query_starts=qs.long()), "query")]:
        with pytest.raises(ValueError, match=what):
            prefill(**kw)
    if torch.cuda.is_available():  # a dtype the library does not store: refused once on a device
        h = lambda t: t.half().cuda()  # noqa: E731
        with pytest.raises(TypeError, match="dtype"):
            npg.np_paged_prefill(h(q), h(q), h(pool), h(pool), bt.cuda(), cl.cuda(), qs.cuda(), 0.1, None)
    with pytest.raises(ValueError, match="cos_sin"):
        npg.prefill_step(q.clone(), q, k, k, slots, pool, pool, bt, cl, qs, 0.1, None, positions=pos)
    with pytest.raises(ValueError, match="rot_dim/2"):
        npg.rope_table(4, 32, inv_freq=[1.0, 0.5], device="cpu")
