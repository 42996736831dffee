"""The expert products' workspace: what a call clears of it, what has to be zero, and which calls a buffer serves."""
import pytest
import torch

import qlora_block_absmax_b200 as nf4
from qlora_block_absmax_b200 import _lib
from tests.test_gpu_experts import activations, check, make_stack, offsets_of, reference

pytestmark = pytest.mark.gpu


def functions(gradient):
    return ((nf4.gemm_experts_dx, nf4.gemm_experts_dx_workspace_bytes) if gradient else
            (nf4.gemm_experts, nf4.gemm_experts_workspace_bytes))


@pytest.mark.parametrize("gradient", [False, True])
def test_a_call_without_a_workspace_clears_the_counters_only(gradient):
    """the block that the call takes from torch's cache was filled before: behind the counters and the partial sums of one
    unit's items the filling is still there"""
    n, k = (1024, 256) if gradient else (256, 1024)
    qw, wc = make_stack(2, n, k, seed=9)
    f, size = functions(gradient)
    off = offsets_of([1, 0])
    x = activations(1, 1024, 23)
    want = f(qw, x, off, 2)
    check(want, *reference(wc, x, off, gradient), 1024)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    need = size(qw, 2, 1)
    filled = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    place = filled.data_ptr()
    del filled
    assert torch.equal(f(qw, x, off, 2), want)
    again = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == place
    assert bool((again[:_lib.NF4_EXPERTS_COUNTER_BYTES] == 0).all())
    assert bool((again[need // 2:] == 0xA5).all())


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("counts", [[1, 0, 0, 0], [2, 2, 2, 2], [33, 0, 0, 40]])
def test_only_the_counters_have_to_be_zero(gradient, counts):
    """NaN everywhere behind the counters: the same bits as with a workspace of zeros, counters zero again afterwards"""
    n, k = (4096, 1024) if gradient else (1024, 4096)
    qw, wc = make_stack(4, n, k)
    f, size = functions(gradient)
    off = offsets_of(counts)
    x = activations(sum(counts), 4096, 24)
    need = size(qw, 4, sum(counts))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:_lib.NF4_EXPERTS_COUNTER_BYTES] = 0
    y = f(qw, x, off, 4, workspace=ws)
    check(y, *reference(wc, x, off, gradient), 4096)
    assert torch.equal(y, f(qw, x, off, 4, workspace=torch.zeros(need, dtype=torch.uint8, device="cuda")))
    assert bool((ws[:_lib.NF4_EXPERTS_COUNTER_BYTES] == 0).all())
    assert torch.equal(y, f(qw, x, off, 4, workspace=ws))
    nf4.check_device_error()


@pytest.mark.parametrize("gradient", [False, True])
def test_a_buffer_sized_for_one_row_serves_every_m(gradient):
    """one buffer, made for a single decoded row, for calls of other numbers of rows in turn"""
    n, k = (4096, 512) if gradient else (512, 4096)
    qw, wc = make_stack(4, n, k)
    f, size = functions(gradient)
    ws = torch.zeros(size(qw, 4, 1), dtype=torch.uint8, device="cuda")
    for counts in ([0, 1, 0, 0], [8, 8, 8, 8], [9, 8, 8, 8], [64, 0, 0, 1], [1, 0, 0, 0], [200, 3, 90, 40], [2, 0, 33, 0]):
        off = offsets_of(counts)
        x = activations(sum(counts), 4096, 25)
        check(f(qw, x, off, 4, workspace=ws), *reference(wc, x, off, gradient), 4096)
    nf4.check_device_error()


@pytest.mark.parametrize("gradient", [False, True])
def test_workspace_refusals(gradient):
    """what is too small, strided or elsewhere"""
    n, k = (1024, 256) if gradient else (256, 1024)
    qw, _ = make_stack(2, n, k, seed=9)
    f, size = functions(gradient)
    off, x = offsets_of([3, 4]), activations(7, 1024, 26)
    need = size(qw, 2, 7)
    ws = torch.zeros(2 * need, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        f(qw, x, off, 2, workspace=ws[:1].expand(need))
    with pytest.raises(ValueError, match="contiguous"):
        f(qw, x, off, 2, workspace=ws[::2])
    with pytest.raises(ValueError, match="device"):
        f(qw, x, off, 2, workspace=ws.cpu())
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        f(qw, x, off, 2, workspace=ws[:need - 16])
    with pytest.raises(RuntimeError, match="MISALIGNED"):
        f(qw, x, off, 2, workspace=ws[1:])
