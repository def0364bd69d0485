"""prefill_step refuses before it writes: what np_paged_prefill would refuse is known before the new
tokens are rotated (in place, by default) and appended, so that a refused step can be called again."""
import pytest
import torch


class _Calls:
    """The library on the CPU: np_paged_prefill_check is its own, launches are only noted."""

    def __init__(self, lib):
        self.lib, self.made = lib, []

    def __getattr__(self, name):
        if name in ("np_paged_prefill_check", "np_status_string"):
            return getattr(self.lib, name)

        def launch(*_):
            self.made.append(name)
            return 0
        return launch


@pytest.fixture()
def npg_on_cpu(monkeypatch):
    from paged_kv_decode_np_gb300 import build_lib
    import paged_kv_decode_np_gb300 as npg
    calls = _Calls(npg.load(build_lib.build()))
    # CPU tensors stand for the current device's: nothing is launched
    monkeypatch.setattr(npg, "load", lambda path=None: calls)
    monkeypatch.setattr(npg, "_device_now", lambda: -1)
    monkeypatch.setattr(npg, "_stream_now", lambda stream, cur: 0)
    return npg, calls


def _args(hq=4, hk=2, d=64, rows=1, n=3, ws_bytes=64 << 20, dtype=torch.float32):
    pool = torch.zeros(2, 4, 16, hk, d, dtype=dtype)
    ws = torch.empty(ws_bytes + 256, dtype=torch.uint8)
    at = -ws.data_ptr() % 256
    return dict(out=torch.zeros(n, hq, d, dtype=dtype), q=torch.ones(n, hq, d, dtype=dtype),
                k_new=torch.ones(n, hk, d, dtype=dtype), v_new=torch.ones(n, hk, d, dtype=dtype),
                slot_mapping=torch.arange(n), k_pool=pool[0], v_pool=pool[1],
                block_tables=torch.zeros(rows, 4, dtype=torch.int32),
                context_lens=torch.full((rows,), n, dtype=torch.int32),
                query_starts=torch.arange(rows + 1, dtype=torch.int32), scale=0.125,
                workspace=ws[at:at + ws_bytes])


ROPE = dict(cos_sin=torch.zeros(9, 64), positions=torch.zeros(3, dtype=torch.int32))


def test_both_calls_are_made_in_order(npg_on_cpu):
    npg, calls = npg_on_cpu
    npg.prefill_step(**_args(), **ROPE)
    assert calls.made == ["np_rope_append_packed", "np_paged_prefill_packed"]


@pytest.mark.parametrize("change,code", [
    (dict(ws_bytes=4096), 3),                # NP_ERR_WORKSPACE: too small
    (dict(hq=18, hk=2), 2),                # NP_ERR_UNSUPPORTED: an fp32 group of 9
    (dict(hq=34, hk=2, dtype=torch.bfloat16), 2),
    (dict(rows=4097), 2),
    (dict(scale=float("nan")), 1),
    (dict(overlap=True), 1),                   # out is q
    (dict(shift=128), 3),                    # misaligned
])
def test_a_refusal_comes_before_the_append(npg_on_cpu, change, code):
    npg, calls = npg_on_cpu
    change = dict(change)
    scale, overlap, shift = (change.pop(k, None) for k in ("scale", "overlap", "shift"))
    a = _args(**change)
    if scale is not None:
        a["scale"] = scale
    if overlap:
        a["out"] = a["q"]
    if shift:
        a["workspace"] = a["workspace"][shift:]
    with pytest.raises(npg.NPError) as e:
        npg.prefill_step(**a, **ROPE)
    assert e.value.status == code
    assert calls.made == []


@pytest.mark.parametrize("key,value", [("query_starts", torch.zeros(3, dtype=torch.int32)),
                                       ("context_lens", torch.zeros(1)),
                                       ("block_tables", torch.zeros(1, 4, dtype=torch.int64)),
                                       ("out", torch.zeros(2, 4, 64))])
def test_the_bindings_own_refusal_comes_before_the_append(npg_on_cpu, key, value):
    npg, calls = npg_on_cpu
    a = _args()
    a[key] = value
    with pytest.raises(ValueError):
        npg.prefill_step(**a, **ROPE)
    assert calls.made == []


def test_check_is_the_calls_own(npg_on_cpu):
    npg, calls = npg_on_cpu
    assert calls.lib.np_paged_prefill_check(None) == 1
    a = _args()
    for k in ("k_new", "v_new", "slot_mapping"):
        del a[k]
    packed = npg._prefill_args(a["out"], a["q"], a["k_pool"], a["v_pool"], a["block_tables"],
                               a["context_lens"], a["query_starts"], a["scale"], a["workspace"], None, None)
    assert calls.lib.np_paged_prefill_check(packed) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rotate", [False, True])
def test_a_refused_step_leaves_everything_and_can_be_called_again(nplib, rotate):
    n, hq, hk, d, bs = 40, 4, 2, 64, 16
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(n, h, d, generator=gen).bfloat16().cuda() for h in (hq, hk, hk))
    kp, vp = torch.randn(2, 4, bs, hk, d, generator=gen).bfloat16().cuda()
    a = dict(k_new=k, v_new=v, slot_mapping=torch.arange(n, device="cuda"),
             block_tables=torch.arange(4, dtype=torch.int32, device="cuda")[None],
             context_lens=torch.tensor([n], dtype=torch.int32, device="cuda"),
             query_starts=torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale=d ** -0.5)
    if rotate:
        a.update(cos_sin=nplib.rope_table(64, d),
                 positions=torch.arange(n, dtype=torch.int32, device="cuda"))
    ws = nplib.prefill_workspace(d)

    def step(w, state):
        nplib.prefill_step(state[0], state[1], k_pool=state[2], v_pool=state[3], workspace=w, **a)
        torch.cuda.synchronize()

    def fresh():
        return [torch.zeros_like(q), q.clone(), kp.clone(), vp.clone()]

    want = fresh()
    step(ws, want)
    got = fresh()
    with pytest.raises(nplib.NPError, match="WORKSPACE"):
        step(ws[:4096], got)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, fresh()))
    step(ws, got)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
