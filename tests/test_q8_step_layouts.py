"""decode_step_q8's new tokens in layouts that are no one run of tokens: what has to be copied is copied on
the call's own stream.  (On the CPU: the library's calls are stubs.)"""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

ROWS, LONGEST, QL, HK, D = 3, 5, 2, 2, 16


class Copies(TorchDispatchMode):
    """The streams that were current when something was copied."""

    def __init__(self, current):
        super().__init__()
        self.current, self.on = current, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if "clone" in str(func) or "copy" in str(func):
            self.on.append(self.current[-1])
        return func(*args, **(kwargs or {}))


@pytest.fixture
def step(monkeypatch):
    import paged_kv_decode_np_gb300 as npg
    current, seen = ["the caller's"], {}

    class Stream:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            current.append(self.s)

        def __exit__(self, *exc):
            current.pop()

    class Library:
        np_paged_decode_q8_check = np_paged_decode_q8_packed = staticmethod(lambda args: 0)

    def append(kp, vp, ks, vs, k, v, slots, err_word, stream):
        seen.update(k=k, v=v, slots=slots)

    monkeypatch.setattr(torch.cuda, "stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("stream", handle))
    monkeypatch.setattr(npg, "_decode_q8_args", lambda *a: b"")
    monkeypatch.setattr(npg, "load", lambda: Library)
    monkeypatch.setattr(npg, "np_kv_append_q8", append)

    def run(k, v, slots, stream):
        with Copies(current) as copies:
            npg.decode_step_q8(None, None, None, None, None, None, None, None, 1.0, None, k_new=k, v_new=v,
                               slot_mapping=slots, stream=stream)
        return seen, copies.on

    return run


def _padded():
    k = torch.arange(ROWS * LONGEST * HK * D, dtype=torch.float32).view(ROWS, LONGEST, HK, D)
    return k[:, :QL], (k + 0.5)[:, :QL], torch.arange(ROWS * LONGEST).view(ROWS, LONGEST)[:, :QL]


def test_slices_of_padded_tokens_are_copied_on_the_calls_stream(step):
    k, v, slots = _padded()
    seen, on = step(k, v, slots, 1234)
    for name, x in (("k", k), ("v", v), ("slots", slots)):
        assert torch.equal(seen[name], x.reshape(ROWS * QL, *x.shape[2:]))
    assert on == [("stream", 1234)] * 3


def test_slices_of_padded_tokens_without_a_stream(step):
    seen, on = step(*_padded(), None)
    assert seen["k"].shape == (ROWS * QL, HK, D) and on == ["the caller's"] * 3


def test_one_run_of_tokens_is_taken_as_it_is(step):
    fused = torch.zeros(ROWS, QL, 3 * HK * D)
    k, v = (fused[..., i * HK * D:(i + 1) * HK * D].unflatten(-1, (HK, D)) for i in (1, 2))
    slots = torch.zeros(ROWS, QL, dtype=torch.int64)
    seen, on = step(k, v, slots, 1234)
    assert on == [] and seen["k"].data_ptr() == k.data_ptr() and seen["v"].data_ptr() == v.data_ptr()
    assert seen["slots"].data_ptr() == slots.data_ptr() and seen["k"].stride(0) == 3 * HK * D
    assert step(k[:, 0], v[:, 0], slots[:, 0].contiguous(), 1234)[1] == []
