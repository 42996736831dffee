"""Products whose reduction has no columns: a sum of nothing is zero, never what the output's memory held."""
import pytest
import torch

import qlora_block_absmax_b200 as nf4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gemv_groups_without_columns_is_zero(dtype):
    gw = nf4.quantize_groups(torch.zeros(20, 0, dtype=dtype, device="cuda"), group=32)
    out = torch.full((3, 20), 7.0, dtype=dtype, device="cuda")
    x = torch.zeros(3, 0, dtype=dtype, device="cuda")
    assert nf4.gemv_groups(gw, x, out=out) is out and bool((out == 0).all())
    filled = torch.full((3, 20), 7.0, dtype=dtype, device="cuda")
    del filled  # a fresh output may take this block
    y = nf4.gemv_groups(gw, x)
    assert y.shape == (3, 20) and bool((y == 0).all())
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        nf4.gemv_groups(gw, torch.zeros(9, 0, dtype=dtype, device="cuda"))
    side = torch.cuda.Stream()
    y = nf4.gemv_groups(gw, x, stream=side)
    side.synchronize()
    assert bool((y == 0).all())


def test_expert_products_without_a_reduction_are_refused():
    """which rows an expert has is known on the GPU only, and the library launches nothing for an empty weight"""
    none = lambda rows, cols: nf4.QuantizedWeight(  # noqa: E731
        packed=torch.zeros(16, dtype=torch.uint8, device="cuda"), rows=rows, cols=cols,
        absmax=torch.zeros(4, device="cuda"))
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    x = torch.zeros(5, 0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="sum over"):
        nf4.gemm_experts(none(256, 0), x, off, 2)
    with pytest.raises(ValueError, match="sum over"):
        nf4.gemm_experts_dx(none(0, 128), x, off, 2)
    # no outputs at all, or no rows: nothing to do
    wide = torch.zeros(5, 128, dtype=torch.bfloat16, device="cuda")
    assert nf4.gemm_experts(none(0, 128), wide, off, 2).shape == (5, 0)
    assert nf4.gemm_experts(none(256, 128), wide[:0], off, 2).shape == (0, 128)
