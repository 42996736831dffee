"""The size of the expert products' workspace (no GPU needed): 0 or one value for every number of rows, so that a buffer
made for one call serves the router's next counts."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

import qlora_block_absmax_b200 as nf4
from qlora_block_absmax_b200 import _lib
from tests.test_abi import weight

ROWS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 255, 512, 513, 1000, 4096, 8192, 100000]


@pytest.mark.parametrize("name", ["nf4_gemm_experts", "nf4_gemm_experts_dx"])
@pytest.mark.parametrize("experts,n,k", [(8, 4096, 4096), (8, 14336, 4096), (64, 1024, 2048), (2, 256, 4096),
                                         (2, 4096, 256), (256, 128, 1024), (1, 1024, 128), (1, 151552, 1024),
                                         (1, 151680, 1024), (1, 1024, 151680)])
def test_one_size_serves_every_number_of_rows(name, experts, n, k):
    lib = _lib.load()
    w = weight(rows=experts * n, cols=k)
    size = getattr(lib, name + "_workspace_bytes")
    sizes = [size(ctypes.byref(w), experts, m) for m in ROWS]
    assert set(sizes) <= {0, sizes[0]}
    red, out = (k, n) if name == "nf4_gemm_experts" else (n, k)
    assert (sizes[0] > 0) == (red >= 1024 and out // 128 <= 8 * 148)
    assert sizes[0] == 0 or sizes[0] >= _lib.NF4_EXPERTS_COUNTER_BYTES + 148 * 64 * 128 * 4


def test_a_strided_workspace_is_refused():
    """an expanded tensor has more elements than memory: its element count says nothing about the bytes behind its start"""
    here = SimpleNamespace(get_device=lambda: 0)

    def buffer(t, cuda=True, device=0):
        return SimpleNamespace(is_cuda=cuda, get_device=lambda: device, is_contiguous=t.is_contiguous, numel=t.numel,
                               element_size=t.element_size)

    whole = torch.zeros(64, dtype=torch.int32)
    assert nf4._workspace_bytes(buffer(whole), here) == 256
    for t in (whole[:1].expand(1 << 24), whole[::2], whole.view(8, 8).t()):
        with pytest.raises(ValueError, match="contiguous"):
            nf4._workspace_bytes(buffer(t), here)
    with pytest.raises(ValueError, match="device"):
        nf4._workspace_bytes(buffer(whole, device=1), here)
    with pytest.raises(ValueError, match="device"):
        nf4._workspace_bytes(buffer(whole, cuda=False), here)
