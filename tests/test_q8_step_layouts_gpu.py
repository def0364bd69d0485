"""decode_step_q8 with new tokens that lie in padded rows, on a stream that is not the current one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ROWS, LONGEST, QL, HK, G, D, BS = 5, 7, 3, 2, 2, 64, 16


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_padded_tokens_while_the_current_stream_is_busy(nplib, handle):
    npg = nplib
    gen = torch.Generator().manual_seed(1)
    i32 = dict(dtype=torch.int32, device="cuda")
    k, v = (torch.randn(ROWS, LONGEST, HK, D, generator=gen).to("cuda", torch.bfloat16) for _ in range(2))
    q = torch.randn(ROWS, QL, HK * G, D, generator=gen).to("cuda", torch.bfloat16)
    tables = torch.arange(ROWS, **i32)[:, None].contiguous()
    lens = torch.full((ROWS,), QL, **i32)
    slots = torch.arange(ROWS, device="cuda")[:, None] * BS + torch.arange(LONGEST, device="cuda")
    ws = npg.decode_q8_workspace(D)
    want_cache, want = npg.q8_pools(ROWS, BS, HK, D), torch.zeros_like(q)
    npg.decode_step_q8(want, q, *want_cache, tables, lens, 0.1, ws, k_new=k[:, :QL].contiguous(),
                       v_new=v[:, :QL].contiguous(), slot_mapping=slots[:, :QL].contiguous())
    cache, out = npg.q8_pools(ROWS, BS, HK, D), torch.zeros_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(1_000_000_000)  # (half a second and more of the current stream)
    busy = torch.cuda.Event()
    busy.record()
    npg.decode_step_q8(out, q, *cache, tables, lens, 0.1, ws, k_new=k[:, :QL], v_new=v[:, :QL],
                       slot_mapping=slots[:, :QL], stream=side.cuda_stream if handle else side)
    side.synchronize()
    assert not busy.query()  # nothing of the step waited for the current stream
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for a, b in zip(cache, want_cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
