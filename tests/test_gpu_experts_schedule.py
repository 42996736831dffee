"""The expert products' schedule on single CTAs: whole units first, then the units of the last round, split."""
import pytest
import torch

import qlora_block_absmax_b200 as nf4
from tests.test_gpu_experts import activations, check, make_stack, offsets_of, reference

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def units(counts, out_cols):
    """tiles of 64 rows x 128 output columns"""
    return sum((c + 63) // 64 for c in counts) * (out_cols // 128)


# out_cols, reduction, rows per expert
MIXED = [
    (2560, 4096, [1, 8, 3, 1, 5, 2, 8, 4]),       # 160 units: a round of whole ones and 12 of 8 items each
    (2944, 4096, [1, 1, 2, 1, 0, 3, 1, 1]),       # 161: the same with an expert without rows
    (2688, 1088, [7, 64, 64, 33, 16, 1, 2, 9]),   # 168, tiles of 64 rows; a reduction of odd length (forward: half a stage)
    (2560, 2112, [17, 0, 65, 30, 66, 3, 31, 1]),  # 180: two row tiles in two experts, their parts in different rounds
    (1152, 1024, [1] * 40),                       # 360: two whole rounds, 64 units left
    (4224, 1024, [2, 1, 0, 5, 1, 9, 12, 1, 4, 4]),  # 297: two whole rounds, one unit left
]


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("case", MIXED, ids=lambda c: f"{c[0]}x{c[1]}x{len(c[2])}")
def test_whole_units_then_split_ones(case, gradient):
    """more units than CTAs and not a multiple: the CTAs go on from whole units to parts of units; one workspace for calls
    in a row, equal bits, another routing in between"""
    out_cols, red, counts = case
    n, k = (red, out_cols) if gradient else (out_cols, red)
    u = units(counts, out_cols)
    assert u > sms() and u % sms() != 0
    qw, wc = make_stack(len(counts), n, k, seed=12)
    f, size = ((nf4.gemm_experts_dx, nf4.gemm_experts_dx_workspace_bytes) if gradient else
               (nf4.gemm_experts, nf4.gemm_experts_workspace_bytes))
    off = offsets_of(counts)
    x = activations(sum(counts), red, 28)
    need = size(qw, len(counts), sum(counts))
    assert need > 0  # (single CTAs, split)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    y = f(qw, x, off, len(counts), workspace=ws)
    check(y, *reference(wc, x, off, gradient), red)
    for _ in range(10):
        assert torch.equal(f(qw, x, off, len(counts), workspace=ws), y)
    other = offsets_of(counts[::-1])
    check(f(qw, x, other, len(counts), workspace=ws), *reference(wc, x, other, gradient), red)
    assert torch.equal(f(qw, x, off, len(counts), workspace=ws), y)
    assert bool((ws[:4096] == 0).all())
    nf4.check_device_error()


@pytest.mark.parametrize("gradient", [False, True])
def test_several_rounds_of_single_ctas(gradient):
    """short reductions, so no workspace: each CTA walks many tiles of several experts on its own"""
    counts = [3, 0, 31, 60, 64, 1, 17, 40] * 4
    out_cols, red = 4352, 192
    n, k = (red, out_cols) if gradient else (out_cols, red)
    qw, wc = make_stack(len(counts), n, k, seed=13)
    assert max(counts) <= 64 and units(counts, out_cols) > 5 * sms()
    f = nf4.gemm_experts_dx if gradient else nf4.gemm_experts
    off = offsets_of(counts)
    x = activations(sum(counts), red, 29)
    y = f(qw, x, off, len(counts))
    check(y, *reference(wc, x, off, gradient), red)
    for _ in range(5):
        assert torch.equal(f(qw, x, off, len(counts)), y)
    nf4.check_device_error()


@pytest.mark.parametrize("gradient", [False, True])
def test_graphs_of_split_calls(gradient):
    """two captured calls, each with its workspace, replayed with another routing each time"""
    out_cols, red, counts = MIXED[0]
    n, k = (red, out_cols) if gradient else (out_cols, red)
    qw, wc = make_stack(len(counts), n, k, seed=12)
    f, size = ((nf4.gemm_experts_dx, nf4.gemm_experts_dx_workspace_bytes) if gradient else
               (nf4.gemm_experts, nf4.gemm_experts_workspace_bytes))
    m = sum(counts)
    off = offsets_of(counts)
    x = activations(m, red, 30)
    ws = torch.zeros(size(qw, len(counts), m), dtype=torch.uint8, device="cuda")
    own, fresh = (torch.zeros(m, out_cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    f(qw, x, off, len(counts), out=own, workspace=ws)
    graphs = []
    for out, w in ((own, ws), (fresh, None)):  # (None: the capture's own buffer, cleared by every replay)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(qw, x, off, len(counts), out=out, workspace=w)
        graphs.append(g)
    for c in (counts, counts[::-1], [m, 0, 0, 0, 0, 0, 0, 0], [0, 0, 0, 1, 0, 0, 0, m - 1]):
        off.copy_(offsets_of(c))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        ref = reference(wc, x, off, gradient)
        check(own, *ref, red)
        assert torch.equal(own, fresh)
    nf4.check_device_error()
