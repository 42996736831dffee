"""Host-side argument checks of the expert products and the group-scale functions: bad arguments are refused before any
CUDA call (no GPU needed)."""
import ctypes

import pytest

from qlora_block_absmax_b200 import _lib
from tests.test_abi import weight

E = {v: k for k, v in _lib.STATUS_NAMES.items()}
BAD, ODD, UNSUP, OK = (E["NF4_ERR_" + n] if n else 0 for n in ("INVALID_ARG", "MISALIGNED", "UNSUPPORTED", ""))


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


@pytest.mark.parametrize("name", ["nf4_gemm_experts", "nf4_gemm_experts_dx"])
def test_experts(lib, name):
    f = lambda w, e=2, x=0x9000, off=0xb000, m=4, y=0xa000, ws=None, n=0: getattr(lib, name)(  # noqa: E731
        ctypes.byref(w) if w is not None else None, e, x, off, m, y, ws, n, None)
    w = weight(rows=256, cols=128)
    assert f(None) == BAD
    assert f(w, e=0) == BAD and f(w, e=257) == BAD and f(w, e=3) == BAD  # 1..256, dividing the rows
    assert f(w, m=-1) == BAD
    assert f(w, x=None) == BAD and f(w, off=None) == BAD and f(w, y=None) == BAD
    assert f(w, x=0x9008) == ODD and f(w, y=0xa008) == ODD and f(w, off=0xb002) == ODD
    assert f(weight(rows=256, cols=128, bs=128)) == UNSUP
    assert f(weight(rows=256, cols=96)) == UNSUP
    assert f(weight(rows=2 * 96, cols=128)) == UNSUP
    # each direction's output tile is 128 wide, its reduction whole blocks of 64
    forward = name == "nf4_gemm_experts"
    assert f(weight(rows=256, cols=192), m=0) == (OK if forward else UNSUP)
    assert f(weight(rows=2 * 192, cols=128), m=0) == (UNSUP if forward else OK)
    assert f(weight(rows=256, cols=128, absmax=0)) == BAD
    assert f(w, m=2 ** 31) == UNSUP  # tensor-map coordinates are 32-bit
    assert f(weight(rows=2 ** 32, cols=128)) == UNSUP
    assert f(w, m=0, x=None, off=None, y=None) == OK  # nothing to compute, nothing launched
    assert f(weight(rows=0, cols=128)) == OK
    size = getattr(lib, name + "_workspace_bytes")
    assert size(None, 2, 4) == 0 and size(ctypes.byref(w), 2, 0) == 0 and size(ctypes.byref(w), 0, 4) == 0


def group_weight(rows=10, cols=128, packed=0x1000, scale=0x2000, zero=0x3001, group=64, dtype=1):
    return _lib.NF4GroupWeight(packed, scale, zero, rows, cols, group, dtype)


def test_groups_weight_rules(lib):
    gemv = lambda w, x=0x9000, b=1, y=0xa000: lib.nf4_gemv_groups(ctypes.byref(w), x, b, y, None)  # noqa: E731
    deq = lambda w, out=0xa000, t=0: lib.nf4_dequantize_groups(ctypes.byref(w), out, t, None)  # noqa: E731
    for f in (gemv, deq):
        assert f(group_weight(group=16)) == UNSUP and f(group_weight(group=256, cols=256)) == UNSUP
        assert f(group_weight(cols=96)) == UNSUP and f(group_weight(group=0)) == UNSUP
        assert f(group_weight(dtype=0)) == BAD and f(group_weight(dtype=3)) == BAD
        assert f(group_weight(rows=-1)) == BAD and f(group_weight(cols=-64)) == BAD
        assert f(group_weight(packed=None)) == BAD and f(group_weight(scale=None)) == BAD
        assert f(group_weight(packed=0x1008)) == ODD and f(group_weight(scale=0x2001)) == ODD
        assert f(group_weight(rows=2 ** 62, cols=2 ** 40)) == BAD
        assert f(group_weight(rows=0)) == OK and f(group_weight(cols=0)) == OK
    w = group_weight()
    assert gemv(w, b=0) == BAD and gemv(w, b=9) == BAD
    assert gemv(w, x=None) == BAD and gemv(w, y=None) == BAD
    assert gemv(w, x=0x9002) == ODD and gemv(w, y=0xa001) == ODD
    assert deq(w, t=5) == BAD and deq(w, out=None) == BAD and deq(w, out=0xa008) == ODD
    assert lib.nf4_gemv_groups(None, 0x9000, 1, 0xa000, None) == BAD
    assert lib.nf4_dequantize_groups(None, 0xa000, 0, None) == BAD


def test_quantize_groups_rules(lib):
    f = lambda src=0x9000, t=0, rows=4, cols=128, g=64, st=1, p=0x1000, s=0x2000, z=0x3000: lib.nf4_quantize_groups(  # noqa: E731
        src, t, rows, cols, g, st, p, s, z, None)
    assert f(t=3) == BAD and f(t=-1) == BAD and f(st=0) == BAD
    assert f(g=48) == UNSUP and f(cols=96) == UNSUP
    assert f(rows=-1) == BAD
    assert f(src=None) == BAD and f(p=None) == BAD and f(s=None) == BAD
    assert f(src=0x9008) == ODD and f(p=0x1004) == ODD and f(s=0x2001) == ODD
    assert f(rows=0, src=None, p=None, s=None, z=None) == OK
