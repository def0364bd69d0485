"""np_paged_prefill's scale: its product with log2(e), which the kernels multiply by, is finite."""
import pytest
import torch


@pytest.mark.parametrize("dtype", [0, 1])
def test_a_scale_whose_product_with_log2e_is_not_finite_is_refused(dtype):
    from paged_kv_decode_np_gb300 import build_lib
    import paged_kv_decode_np_gb300 as npg
    lib = npg.load(build_lib.build())
    at = [0x100000 * (i + 1) for i in range(4)]

    def check(scale):
        return lib.np_paged_prefill_check(npg._PREFILL_ARGS.pack(
            *at, at[0], at[0], at[0], 0x10000000, 0, 0, 16, 1 << 30, dtype, 16, 2, 128, 4, 2, 5, 4, scale))

    for scale in (0.0, 0.1, -0.1, 1e-38, 2.3e38, -2.3e38):
        assert check(scale) == 0, scale
    for scale in (2.4e38, -2.4e38, 3.4e38, 1e39, float("inf"), float("nan")):
        assert check(scale) == 1, scale


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 256), (torch.float32, 64),
                                     (torch.float32, 256)])
@pytest.mark.parametrize("scale", [2.0 ** 31, -2.0 ** 31, 0.0, 1e-38])
def test_extreme_scales(nplib, dtype, d, scale):
    """Large: all weight on the largest score (the smallest).  Small: equal weights."""
    n, c, hk, g, bs = 4, 150, 2, 2, 16
    gen = torch.Generator().manual_seed(d)
    q = torch.zeros(n, hk * g, d)
    q[..., 0] = 0.125  # |scale q.k| < 2^29
    nb = -(-c // bs)
    # distinct scores of a few bits: what exceeds a score by 2^-10 outweighs it by e^(2^21)
    k, v = torch.zeros(nb * bs, hk, d), torch.randn(nb * bs, hk, d, generator=gen).to(dtype).float()
    order = torch.randperm(c, generator=gen)
    k[:c, :, 0] = (1 + order.float() / 128)[:, None].clamp(max=1.9921875) if scale else 1.0
    k[:c][order >= 127, :, 0] = 0.5 if scale > 0 else 1.9921875  # the rest: never the extreme one
    out = torch.zeros(n, hk * g, d, dtype=dtype, device="cuda")
    put = lambda x: x.to(dtype).cuda()  # noqa: E731
    nplib.np_paged_prefill(out, put(q), put(k.view(nb, bs, hk, d)), put(v.view(nb, bs, hk, d)),
                           torch.arange(nb, dtype=torch.int32, device="cuda")[None],
                           torch.tensor([c], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale,
                           nplib.prefill_workspace(d))
    torch.cuda.synchronize()
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24  # half a step
    for i in range(n):
        seen = c - n + i + 1
        vi = v[:seen].double()
        if abs(scale) > 1:
            s = k[:seen, 0, 0].double() * (1 if scale > 0 else -1)
            assert (s == s.max()).sum() == 1
            # one weight, rounded for its product with v, over itself; the result rounded once
            want = vi[s.argmax()]
            tol = 4 * half * want.abs()
        else:
            want = vi.mean(0)
            # equal weights of 1: exact in bf16; sums and the quotient as fp32 sums; one rounding
            tol = 2 * c * 2.0 ** -23 * vi.abs().mean(0) + half * want.abs()
        got = out[i].cpu().double().view(hk, g, d)
        assert ((got - want[:, None]).abs() <= tol[:, None]).all()
