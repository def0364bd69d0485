"""np_paged_prefill with a negative scale on every kernel: the sign is the matrix products' (bf16; fp32 to
head_dim 128) or the multiplication's after them (fp32 at head_dim 256)."""
import pytest
import torch

from prompt_helpers import chunk_inputs, chunk_reference, chunk_tolerance

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,d,bs", [(F32, 256, 16), (F32, 128, 16), (F32, 16, 8), (BF, 128, 16), (BF, 128, 5),
                                        (BF, 256, 16), (BF, 32, 16)])
@pytest.mark.parametrize("scale", [-0.2, -0.02])
def test_negative_scales(nplib, dtype, d, bs, scale):
    rows = [(20, 90), (130, 330), (1, 500), (9, 5)]
    inp = chunk_inputs(dtype, d, 2, 3, bs, rows, seed=d)
    out, err = torch.empty_like(inp["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    nplib.np_paged_prefill(out, inp["q"], inp["k_pool"], inp["v_pool"], inp["block_tables"],
                           inp["context_lens"], inp["query_starts"], scale, nplib.prefill_workspace(d),
                           err_word=err)
    torch.cuda.synchronize()
    ref, bound = chunk_reference(inp, rows, scale)
    assert int(err) == 0
    assert ((out.double() - ref).abs() <= chunk_tolerance(ref, bound, dtype, d, 500)).all()
