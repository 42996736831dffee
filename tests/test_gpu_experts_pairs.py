"""The expert products on CTA pairs, against fp64 sums over the oracle's 16-bit weights (tolerance: see check)."""
import ctypes

import pytest
import torch

import qlora_block_absmax_b200 as nf4
from qlora_block_absmax_b200 import _lib
from tests.test_gpu_experts import activations, check, make_stack, offsets_of, reference

pytestmark = pytest.mark.gpu

COUNTS = [257, 1, 0, 130, 512, 31, 700, 256]


def takes_pairs(qw, experts, x, off, gradient):
    """Whether the call runs on CTA pairs: with a reduction this long and tiles this few, a call on single CTAs needs a
    workspace for its split reductions and is refused without one."""
    out_cols, red = (qw.cols, qw.rows // experts) if gradient else (qw.rows // experts, qw.cols)
    m = x.shape[0]
    assert red >= 1024 and (m + 63) // 64 * (out_cols // 128) <= 8 * 148
    lib = _lib.load()
    f = lib.nf4_gemm_experts_dx if gradient else lib.nf4_gemm_experts
    y = torch.empty(m, out_cols, dtype=torch.bfloat16, device="cuda")
    d = qw.descriptor()
    st = f(ctypes.byref(d), experts, x.data_ptr(), off.data_ptr(), m, y.data_ptr(), None, 0,
           torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert _lib.STATUS_NAMES[st] in ("NF4_OK", "NF4_ERR_INVALID_ARG")
    return st == 0


def run_pairs(qw, wc, out_cols, red, gradient, seed, repeats):
    off = offsets_of(COUNTS, lead=3)
    x = activations(sum(COUNTS) + 5, red, seed)
    f = nf4.gemm_experts_dx if gradient else nf4.gemm_experts
    if red >= 1024:
        assert takes_pairs(qw, len(COUNTS), x, off, gradient)
    out = torch.full((x.shape[0], out_cols), 3.5, dtype=torch.bfloat16, device="cuda")
    f(qw, x, off, len(COUNTS), out=out)
    check(out, *reference(wc, x, off, gradient), red)
    assert bool((out[:3] == 3.5).all()) and bool((out[-2:] == 3.5).all())
    for _ in range(repeats):
        assert torch.equal(f(qw, x, off, len(COUNTS), out=out.clone()), out)
    nf4.check_device_error()


@pytest.mark.parametrize("out_cols", [1408, 2048, 2176])
@pytest.mark.parametrize("red", [1024, 1088, 2560])
def test_gradient_hand_over(out_cols, red):
    """the decoded tile of CTA 1 goes to an MMA that CTA 0 issues: every output against fp64, equal bits on many calls"""
    qw, wc = make_stack(len(COUNTS), red, out_cols, seed=8)
    run_pairs(qw, wc, out_cols, red, True, 22, 40)


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("scales", ["plain", "e4m3", "int8"])
@pytest.mark.parametrize("book", ["nf4", "fp4"])
@pytest.mark.parametrize("out_cols,red", [(2176, 1024), (2048, 1088), (1792, 1024), (2176, 192)])
def test_weight_forms_on_pairs(book, scales, gradient, out_cols, red):
    """every kind of weight on CTA pairs.  Widths with and without a last column tile of 128; rows of scales that are whole
    16-byte units and that are not, by the output's width (gradient: 2048 both, 1792 the fp32 scales only) and by the
    reduction's (forward: 1024 codes 16 at a time)"""
    n, k = (red, out_cols) if gradient else (out_cols, red)
    qw, wc = make_stack(len(COUNTS), n, k, book, scales, seed=11)
    run_pairs(qw, wc, out_cols, red, gradient, 27, 3)
