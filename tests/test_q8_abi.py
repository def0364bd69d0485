"""The 8-bit cache's refusals, on the CPU: every call here fails validation or has nothing to do before
anything touches a device."""
import pytest
import torch

FAKE = 0x1000000  # an aligned address that is never dereferenced
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from paged_kv_decode_np_gb300 import build_lib
    path = build_lib.build()
    import paged_kv_decode_np_gb300 as npg
    return npg.load(path)


def _map(lib, **kw):
    import paged_kv_decode_np_gb300 as npg
    a = dict(tables=FAKE, lens=FAKE + MB, new=FAKE + 2 * MB, kept=None, free=FAKE + 3 * MB, count=FAKE + 4 * MB,
             starts=FAKE + 5 * MB, slots=FAKE + 6 * MB, pos=FAKE + 7 * MB, err=None, nb=64, mb=8, rows=4, bs=16, n=10)
    a.update(kw)
    return lib.np_block_map_packed(npg._MAP_ARGS.pack(
        *[a[k] or 0 for k in ("tables", "lens", "new", "kept", "free", "count", "starts", "slots", "pos", "err")],
        0, a["nb"], a["mb"], a["rows"], a["bs"], a["n"]))


def test_block_map_refusals(lib):
    assert lib.np_block_map_packed(None) == 1
    assert _map(lib, rows=0, n=0) == 0
    assert _map(lib, rows=0, n=0, starts=None) == 0
    for name in ("tables", "lens", "new", "free", "count", "starts", "slots"):
        assert _map(lib, **{name: None}) == 1, name
        assert _map(lib, **{name: FAKE + 3}) == 1, name
    assert _map(lib, n=0) == 1                          # a slot mapping of no tokens
    assert _map(lib, slots=None, n=0) == 1              # positions without slots
    assert _map(lib, rows=-1) == 1
    assert _map(lib, n=-1) == 1
    assert _map(lib, bs=0) == 1
    assert _map(lib, mb=0) == 1
    assert _map(lib, nb=0) == 1
    assert _map(lib, rows=4097) == 2
    assert _map(lib, mb=2**28, bs=16) == 2              # positions past int32
    assert _map(lib, rows=4096, mb=2**20, bs=1) == 2    # blocks past int32
    assert _map(lib, nb=2**32) == 2
    assert _map(lib, nb=2**62) == 4
    assert _map(lib, slots=FAKE + 6 * MB + 4) == 1
    assert _map(lib, lens=FAKE + 64) == 1               # inside the tables
    assert _map(lib, new=FAKE + MB) == 1                # the lengths themselves
    assert _map(lib, kept=FAKE + MB + 4) == 1           # context_lens, shifted
    assert _map(lib, starts=FAKE + 3 * MB) == 1
    assert _map(lib, pos=FAKE + 6 * MB) == 1


def _append(lib, **kw):
    import paged_kv_decode_np_gb300 as npg
    a = dict(kp=FAKE, vp=FAKE + MB, ks=FAKE + 2 * MB, vs=FAKE + 3 * MB, k=FAKE + 4 * MB, v=FAKE + 5 * MB,
             sm=FAKE + 6 * MB, err=None, nb=16, kst=256, vst=256, form=0, dtype=1, bs=16, hk=2, d=128, n=3)
    a.update(kw)
    return lib.np_kv_append_q8_packed(npg._APPEND_Q8_ARGS.pack(
        *[a[k] or 0 for k in ("kp", "vp", "ks", "vs", "k", "v", "sm", "err")], 0, a["nb"], a["kst"], a["vst"],
        a["form"], a["dtype"], a["bs"], a["hk"], a["d"], a["n"]))


def test_append_refusals(lib):
    assert lib.np_kv_append_q8_packed(None) == 1
    assert _append(lib, n=0) == 0
    for name in ("kp", "vp", "ks", "vs", "k", "v", "sm"):
        assert _append(lib, **{name: None}) == 1, name
        assert _append(lib, **{name: FAKE + 8 * MB + 2}) == 1, name
    assert _append(lib, kp=FAKE + 8 * MB + 4) == 1
    assert _append(lib, hk=4097) == 2
    assert _append(lib, n=-1) == 1
    assert _append(lib, form=2) == 2
    assert _append(lib, dtype=2) == 2
    assert _append(lib, d=96) == 2
    assert _append(lib, hk=0) == 1
    assert _append(lib, nb=0) == 1
    assert _append(lib, bs=0) == 1
    assert _append(lib, nb=2**62) == 4
    assert _append(lib, kst=255) == 1                   # tokens run into one another
    assert _append(lib, vst=260) == 1                   # not a multiple of 16 bytes
    assert _append(lib, kst=-256) == 1
    assert _append(lib, kst=2**61, n=100) == 4
    assert _append(lib, vp=FAKE + 64) == 1              # one pool in the other
    assert _append(lib, ks=FAKE + 64) == 1
    assert _append(lib, k=FAKE + 1024) == 1             # the new tokens in a pool
    assert _append(lib, sm=FAKE + 3 * MB + 16) == 1     # the slots in the scales


def _read(lib, call="np_paged_decode_q8_packed", **kw):
    import paged_kv_decode_np_gb300 as npg
    prefill = "prefill" in call
    a = dict(out=FAKE, q=FAKE + MB, kp=FAKE + 2 * MB, vp=FAKE + 3 * MB, ks=FAKE + 4 * MB, vs=FAKE + 5 * MB,
             bt=FAKE + 6 * MB, cl=FAKE + 7 * MB, qst=FAKE + 8 * MB if prefill else None, ws=FAKE + 16 * MB, err=None,
             nb=16, wsb=64 << 20, form=0, dtype=1, bs=16, hk=2, d=128, mb=4, rows=2, ql=0 if prefill else 1, n=2,
             hq=4, scale=0.1)
    a.update(kw)
    return getattr(lib, call)(npg._READ_Q8_ARGS.pack(
        *[a[k] or 0 for k in ("out", "q", "kp", "vp", "ks", "vs", "bt", "cl", "qst", "ws", "err")], 0, a["nb"],
        a["wsb"], a["form"], a["dtype"], a["bs"], a["hk"], a["d"], a["mb"], a["rows"], a["ql"], a["n"], a["hq"],
        a["scale"]))


@pytest.mark.parametrize("call", ["np_paged_decode_q8_packed", "np_paged_decode_q8_check",
                                  "np_paged_prefill_q8_packed", "np_paged_prefill_q8_check"])
def test_read_refusals(lib, call):
    def read(**kw):
        return _read(lib, call, **kw)

    prefill = "prefill" in call
    assert getattr(lib, call)(None) == 1
    assert read(rows=0) == 0
    for name in ("out", "q", "kp", "vp", "ks", "vs", "bt", "cl") + (("qst",) if prefill else ()):
        assert read(**{name: None}) == 1, name
        assert read(**{name: FAKE + 9 * MB + 2}) == 1, name
    assert read(ws=None) == 3
    assert read(ws=FAKE + 16 * MB + 16) == 3
    assert read(wsb=1 << 20) == 3
    assert read(rows=-1) == 1
    assert read(form=2) == 2
    assert read(form=-1) == 2
    assert read(dtype=2) == 2
    assert read(d=48) == 2
    assert read(hq=3) == 1                              # not a multiple of the kv heads
    assert read(hq=34) == 2                             # 17 heads a kv head
    assert read(hq=18, dtype=0) == 2                    # fp32: 9
    assert read(scale=float("nan")) == 1
    assert read(scale=3e38) == 1
    assert read(nb=2**62) == 4
    assert read(mb=2**30, bs=16) == 2
    assert read(out=FAKE + MB + 512) == 1               # out in q
    assert read(out=FAKE + 2 * MB + 512) == 1
    assert read(out=FAKE + 4 * MB) == 1                 # in the scales
    if prefill:
        assert read(ql=1) == 1
        assert read(n=0) == 0
        assert read(rows=4097) == 2
    else:
        assert read(ql=0) == 1
        assert read(ql=9) == 2                          # 18 rows
        assert read(ql=5, dtype=0) == 2
        assert read(rows=65536) == 2
        assert read(rows=60000, mb=2**26, bs=16) == 2   # more positions than a block can count


def test_workspaces(lib):
    import paged_kv_decode_np_gb300 as npg
    for d in (16, 32, 64, 128, 256):
        assert 0 < npg.np_paged_decode_q8_workspace_bytes(d) <= npg.NP_DECODE_Q8_WORKSPACE_BYTES
    assert npg.np_paged_decode_q8_workspace_bytes(48) == 0


def test_binding_refuses_shapes_and_types(lib):
    import paged_kv_decode_np_gb300 as npg
    kp, vp, ks, vs = npg.q8_pools(4, 16, 2, 64, device="cpu")
    k = torch.zeros(3, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        npg.q8_pools(4, 16, 2, 64, torch.float16, device="cpu")
    with pytest.raises(TypeError):
        npg.np_kv_append_q8(kp.float(), vp.float(), ks, vs, k, k, slots)
    with pytest.raises(TypeError):
        npg.np_kv_append_q8(kp, vp.view(torch.int8), ks, vs, k, k, slots)
    with pytest.raises(ValueError):
        npg.np_kv_append_q8(kp, vp, ks[:3], vs, k, k, slots)
    with pytest.raises(ValueError):
        npg.np_kv_append_q8(kp, vp, ks, vs.double(), k, k, slots)
    with pytest.raises(ValueError):
        npg.np_kv_append_q8(kp, vp, ks, vs, k[:, :1], k[:, :1], slots)
    with pytest.raises(ValueError):
        npg.np_kv_append_q8(kp, vp, ks, vs, k, k.bfloat16(), slots)
    with pytest.raises(ValueError):
        npg.np_kv_append_q8(kp, vp, ks, vs, k, k, slots.int())
    with pytest.raises(ValueError, match="CUDA"):
        npg.np_kv_append_q8(kp, vp, ks, vs, k, k, slots)
    q, tab, lens = torch.zeros(3, 4, 64), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(q=torch.zeros(3, 4, 32)), dict(out=torch.zeros(3, 4, 64).bfloat16()), dict(tab=tab.long()),
                dict(tab=tab[:2]), dict(lens=lens[:2]), dict()):
        a = dict(q=q, out=torch.zeros_like(q), tab=tab, lens=lens)
        a.update(bad)
        if "q" in bad:
            a["out"] = torch.zeros_like(bad["q"])
        with pytest.raises(ValueError):
            npg.np_paged_decode_q8(a["out"], a["q"], kp, vp, ks, vs, a["tab"], a["lens"], 0.1, None)
    with pytest.raises(ValueError):
        npg.np_paged_prefill_q8(q, q, kp, vp, ks, vs, tab, lens, None, 0.1, None)
    with pytest.raises(ValueError):
        npg.np_paged_prefill_q8(q, q, kp, vp, ks, vs, tab, lens, lens, 0.1, None)
    one = torch.zeros(1, dtype=torch.int32)
    starts = torch.zeros(4, dtype=torch.int32)
    for bad in (dict(new=lens[:2]), dict(kept=lens.long()), dict(starts=lens), dict(count=lens), dict(pos=starts),
                dict(slots=None), dict()):
        a = dict(new=lens, kept=lens, starts=starts, count=one, slots=slots, pos=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            npg.np_block_map(tab, lens, a["new"], lens, a["count"], a["starts"], a["slots"], a["pos"], 16,
                             kept_lens=a["kept"])
