"""Weights of uniform 4-bit codes with group scales: quantize_groups bit for bit against the definition in numpy (fp32
steps, each rounded once), dequantize_groups bit for bit, gemv_groups against fp64 sums.

gemv_groups tolerance, per output: half a step of the output type (finfo.eps / 2 relative; half the smallest step of
fp16 absolute) plus the fp32 sums' error.  Every product (q - z) x is exact in fp32; an MMA adds 16 of them to the running sum with at
most 17 roundings or truncations, each below 2^-23 of the largest partial sum, which never exceeds the sum of absolute
values S of the group; then one product and one sum per group and 8 sums across warps: in all below
(K / 16 * 17 + 2 K / G + 8) * 2^-23 * S <= (K * 9 / 8 + 8) * 2^-23 * S for G >= 32."""
import numpy as np
import pytest
import torch

import qlora_block_absmax_b200 as nf4
from qlora_block_absmax_b200 import synth

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def quantize_ref(w32, group, symmetric, dtype):
    """(codes, scale as a torch tensor, zero points) of fp32 values, by the definition"""
    n, k = w32.shape
    g = w32.reshape(n, k // group, group)
    if symmetric:
        s = (np.abs(g).max(2) / np.float32(7)).astype(np.float32)
    else:
        lo, hi = np.minimum(g.min(2), 0), np.maximum(g.max(2), 0)
        s = ((hi - lo).astype(np.float32) / np.float32(15)).astype(np.float32)
    st = torch.from_numpy(np.minimum(s, np.float32(torch.finfo(dtype).max))).to(dtype)
    sf = st.float().numpy()
    safe = np.where(sf > 0, sf, np.float32(1))
    z = np.full_like(sf, 8) if symmetric else np.where(sf > 0, np.minimum(np.rint(-lo / safe), 15), 0)
    q = np.clip(np.rint(g / safe[..., None]) + z[..., None], 0, 15)
    q = np.where(sf[..., None] > 0, q, z[..., None])
    return q.astype(np.uint8).reshape(n, k), st, z.astype(np.uint8)


def pack_ref(q):
    n, k = q.shape
    c = q.reshape(n, k // 8, 8).astype(np.uint32)
    word = sum(c[..., j] << np.uint32(4 * (j // 2) + 16 * (j % 2)) for j in range(8)).astype("<u4")
    return word.view(np.uint8).reshape(n, k // 2)


def values_ref(q, st, z, group):
    n, k = q.shape
    v = (q.reshape(n, k // group, group).astype(np.float64) - z[..., None]) * st.double().numpy()[..., None]
    return v.reshape(n, k)


def group_weights(rows, cols, seed):
    """normal weights with hand-made rows: zeros, signed zeros, one sign only, constants, exact ties, tiny values"""
    w = synth.normal_weights((rows, cols), seed)
    if rows >= 8:
        w[0] = 0.0
        w[1] = -0.0
        w[2] = np.abs(w[2])
        w[3] = -np.abs(w[3])
        w[4] = np.float32(0.25)
        w[5] = (np.arange(cols) % 31 - 15) * np.float32(0.5)  # half steps of a scale of 1 (15 / 15 ..) and ties
        w[6] *= np.float32(1e-36)
        w[7] *= np.float32(1e-39)
    return w


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("src", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,ngroups", [(1, 1), (9, 3), (131, 5), (257, 32)])
def test_quantize_groups_bits(group, symmetric, src, rows, ngroups):
    cols = group * ngroups
    w = torch.from_numpy(group_weights(rows, cols, 40 + rows + group)).to(TYPES[src])
    for dtype in (torch.bfloat16, torch.float16):
        gw = nf4.quantize_groups(w.cuda(), group, symmetric, dtype)
        q, st, z = quantize_ref(w.float().numpy(), group, symmetric, dtype)
        assert torch.equal(gw.scale.cpu().view(torch.int16), st.view(torch.int16))
        if symmetric:
            assert gw.zero is None
        else:
            assert np.array_equal(gw.zero.cpu().numpy(), z)
        assert np.array_equal(gw.packed.cpu().numpy(), pack_ref(q))
        v = torch.from_numpy(values_ref(q, st, z, group))
        for out in TYPES.values():
            got = nf4.dequantize_groups(gw, out).cpu()
            assert torch.equal(got.double(), v.float().to(out).double())  # the value is exact in fp32


def random_weight(rows, cols, group, dtype, zeros, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda hi, shape: torch.randint(0, hi, shape, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    packed = r(256, (rows, cols // 2)).to(torch.uint8)
    scale = (torch.rand(rows, cols // group, generator=g, device="cuda") * 0.02 + 0.001).to(dtype)
    zero = r(16, (rows, cols // group)).to(torch.uint8) if zeros else None
    return nf4.GroupWeight(packed=packed, scale=scale, zero=zero, rows=rows, cols=cols, group=group)


def weight_values(gw):
    """fp64 [rows, cols] on the GPU, from the packed words by the definition"""
    b = gw.packed.reshape(gw.rows, gw.cols // 8, 4).long()
    word = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24
    q = torch.stack([(word >> (4 * (j // 2) + 16 * (j % 2))) & 15 for j in range(8)], -1)
    q = q.reshape(gw.rows, gw.cols // gw.group, gw.group).double()
    z = gw.zero.double()[..., None] if gw.zero is not None else 8.0
    return ((q - z) * gw.scale.double()[..., None]).reshape(gw.rows, gw.cols)


def check_gemv(gw, x, y):
    w, xd = weight_values(gw), x.reshape(-1, gw.cols).double()
    ref, s = xd @ w.t(), xd.abs() @ w.abs().t()
    fi = torch.finfo(x.dtype)
    tol = ref.abs() * fi.eps / 2 + fi.tiny * fi.eps + (gw.cols * 9 / 8 + 8) * 2.0 ** -23 * s * (1 + fi.eps)
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,rows,cols", [(32, 1, 32), (32, 17, 96), (32, 100, 4128), (64, 16, 64), (64, 31, 192),
                                             (64, 1000, 1088), (128, 5, 128), (128, 48, 384), (128, 2049, 4096),
                                             (128, 33, 14336), (32, 64, 20000)])
def test_gemv_groups(dtype, zeros, group, rows, cols):
    gw = random_weight(rows, cols, group, dtype, zeros, rows + cols)
    g = torch.Generator(device="cuda").manual_seed(7)
    for batch in (1, 2, 3, 5, 8):
        x = torch.randn(batch, cols, generator=g, device="cuda").to(dtype)
        check_gemv(gw, x, nf4.gemv_groups(gw, x))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemv_groups_one_hot_is_the_weight(group):
    """a one-hot x gives the weight's column, each value rounded once; all other rows of x are zero"""
    gw = random_weight(40, 256, group, torch.bfloat16, True, 3)
    w = weight_values(gw)
    for k in list(range(0, 256, 17)) + [255]:
        x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
        x[1, k] = 1.0
        y = nf4.gemv_groups(gw, x)
        assert torch.equal(y[1].double(), w[:, k].float().bfloat16().double())
        assert bool((y[0] == 0).all())


def test_gemv_groups_rows_of_x_do_not_mix():
    """an Inf and a NaN in one row of x stay in that row's outputs"""
    gw = random_weight(50, 512, 64, torch.bfloat16, False, 4)
    x = torch.randn(4, 512, device="cuda").bfloat16()
    clean = nf4.gemv_groups(gw, x)
    x[2, 5], x[3, 500] = float("inf"), float("nan")
    y = nf4.gemv_groups(gw, x)
    assert torch.equal(y[:2], clean[:2])
    assert bool(torch.isnan(y[3]).all())


def test_gemv_groups_zero_points_cancel_exactly():
    """codes equal to their zero point give exact zeros, whatever x"""
    rows, cols, group = 37, 640, 32
    zero = torch.randint(0, 16, (rows, cols // group), device="cuda", dtype=torch.int32).to(torch.uint8)
    byte = (zero | zero << 4).repeat_interleave(group // 2, 1).contiguous()
    gw = nf4.GroupWeight(packed=byte, scale=torch.ones(rows, cols // group, dtype=torch.bfloat16, device="cuda"),
                         zero=zero, rows=rows, cols=cols, group=group)
    x = (torch.randn(8, cols, device="cuda") * 1e4).bfloat16()
    assert bool((nf4.gemv_groups(gw, x) == 0).all())


def test_gemv_groups_writes_its_rows_only():
    gw = random_weight(19, 128, 128, torch.bfloat16, True, 5)
    buf = torch.full((3 * 19 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(3, 128, device="cuda").bfloat16()
    out = buf[:57].view(3, 19)
    nf4.gemv_groups(gw, x, out=out)
    check_gemv(gw, x, out)
    assert bool((buf[57:] == 7.0).all())


def test_gemv_groups_unaligned_meta_and_stream_and_graph():
    """scales and zero points at odd addresses; a side stream; capture and replay on new inputs"""
    base = random_weight(64, 512, 32, torch.float16, True, 6)
    s = torch.empty(base.scale.numel() + 1, dtype=torch.float16, device="cuda")[1:].view_as(base.scale)
    z = torch.empty(base.zero.numel() + 3, dtype=torch.uint8, device="cuda")[3:].view_as(base.zero)
    s.copy_(base.scale)
    z.copy_(base.zero)
    gw = nf4.GroupWeight(packed=base.packed, scale=s, zero=z, rows=64, cols=512, group=32)
    x = torch.randn(2, 512, device="cuda").half()
    want = nf4.gemv_groups(base, x)
    assert torch.equal(nf4.gemv_groups(gw, x), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = nf4.gemv_groups(gw, x)
    side.synchronize()
    assert torch.equal(y, want)
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(graph):
        nf4.gemv_groups(gw, x, out=out)
    for _ in range(2):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, nf4.gemv_groups(base, x))


def test_quantize_groups_ties():
    """16-bit weights on a grid of half steps of their scale: nearly every quotient is a tie, rounded to even as the
    division would"""
    g = np.random.default_rng(9)
    for dtype in (torch.bfloat16, torch.float16):
        for group in (32, 128):
            steps = g.integers(-15, 16, (64, 512)).astype(np.float32)  # half steps: -7.5 .. 7.5
            steps.reshape(64, -1, group)[:, :, 0], steps.reshape(64, -1, group)[:, :, 1] = -15, 15
            w = torch.from_numpy(steps * np.float32(0.5) * g.choice([2.0 ** -6, 3 * 2.0 ** -9, 2.0 ** -3], (64, 1)).astype(
                np.float32)).to(dtype)
            for symmetric in (False, True):
                gw = nf4.quantize_groups(w.cuda(), group, symmetric)
                q, st, z = quantize_ref(w.float().numpy(), group, symmetric, dtype)
                assert torch.equal(gw.scale.cpu(), st)
                assert np.array_equal(gw.packed.cpu().numpy(), pack_ref(q))
                assert symmetric or np.array_equal(gw.zero.cpu().numpy(), z)


def test_groups_side_stream_argument():
    w = torch.randn(64, 256, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    gw = nf4.quantize_groups(w, 64, stream=side)
    v = nf4.dequantize_groups(gw, stream=side)
    x = torch.ones(2, 256, dtype=torch.bfloat16, device="cuda")
    torch.cuda.current_stream().synchronize()
    y = nf4.gemv_groups(gw, x, stream=side)
    side.synchronize()
    assert torch.equal(v.double(), weight_values(gw))
    check_gemv(gw, x, y)


def test_quantize_groups_then_product():
    """a weight through quantize, its values and the decode product: the product uses exactly the expanded values"""
    w = torch.from_numpy(group_weights(300, 1024, 77)).cuda()
    for dtype in (torch.bfloat16, torch.float16):
        for symmetric in (False, True):
            gw = nf4.quantize_groups(w, 64, symmetric, dtype)
            assert torch.equal(weight_values(gw), nf4.dequantize_groups(gw).double())
            x = torch.randn(4, 1024, device="cuda").to(dtype)
            check_gemv(gw, x, nf4.gemv_groups(gw, x))


def test_groups_refusals():
    w = torch.zeros(4, 96, device="cuda")
    for call in (lambda: nf4.quantize_groups(w, 64), lambda: nf4.quantize_groups(w, 48),
                 lambda: nf4.quantize_groups(w.reshape(-1)), lambda: nf4.quantize_groups(w.cpu()),
                 lambda: nf4.quantize_groups(w.t(), 32)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        nf4.quantize_groups(w.double(), 32)
    with pytest.raises(TypeError):
        nf4.quantize_groups(w, 32, scale_dtype=torch.float32)
    gw = nf4.quantize_groups(w, 32)
    x = torch.zeros(1, 96, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        nf4.gemv_groups(gw, x.half())
    with pytest.raises(ValueError):
        nf4.gemv_groups(gw, x[:, :64].contiguous())
    with pytest.raises(ValueError):
        nf4.gemv_groups(gw, x, out=torch.zeros(1, 5, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        nf4.gemv_groups(gw, x.repeat(9, 1))
    with pytest.raises(TypeError):
        nf4.dequantize_groups(gw, torch.float64)
    assert nf4.quantize_groups(w[:0], 32).packed.numel() == 0
