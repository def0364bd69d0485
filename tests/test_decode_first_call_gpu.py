"""The decode read's first call of a host thread, which has launched nothing before it."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [0, 1, 4])
def test_a_new_host_threads_first_read(nplib, splits):
    rows, hq, hk, d, bs, mb = 3, 8, 8, 128, 16, 20
    gen = torch.Generator().manual_seed(splits)
    kp, vp = (torch.randn(rows * mb, bs, hk, d, generator=gen).bfloat16().cuda() for _ in range(2))
    q = torch.randn(rows, hq, d, generator=gen).bfloat16().cuda()
    bt = torch.arange(rows * mb, dtype=torch.int32, device="cuda").view(rows, mb)
    cl = torch.tensor([320, 17, 100], dtype=torch.int32, device="cuda")
    ws = [nplib.workspace(rows, hq, d, splits) for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(3)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def read(out, w, stream=None):
        nplib.decode_step(out, q, kp, vp, bt, cl, d ** -0.5, num_splits=splits, workspace=w, stream=stream)

    bad = []

    def work():
        try:
            read(outs[1], ws[1], s)
            read(outs[2], ws[1], s)  # and its second
        except BaseException as e:
            bad.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not bad, bad
    read(outs[0], ws[0])
    torch.cuda.synchronize()
    assert torch.equal(outs[1], outs[0]) and torch.equal(outs[2], outs[0])
