"""The products grouped by expert (gemm_experts, gemm_experts_dx) against fp64 sums over the oracle's 16-bit weights.

Tolerance, per output: half a bf16 step (2^-8 relative) plus the fp32 sums' error: the products of two bf16 are exact in
fp32, an MMA adds 16 of them to the running sum with at most 17 roundings or truncations, each below 2^-23 of a partial
sum that never exceeds the sum of absolute values S, so R terms err by less than (17 R / 16 + 8) * 2^-23 * S (the 8: the
partial sums of a split reduction, at most 8 of them)."""
import numpy as np
import pytest
import torch

import oracle
import qlora_block_absmax_b200 as nf4
from qlora_block_absmax_b200 import synth

pytestmark = pytest.mark.gpu


def make_stack(experts, n, k, book="nf4", scales="e4m3", seed=0):
    """(QuantizedWeight of the stack, its 16-bit weights as fp64 [experts, n, k] on the GPU)"""
    w = synth.normal_weights((experts * n, k), 500 + seed)
    quant = oracle.fp4_quantize if book == "fp4" else oracle.quantize
    deq = oracle.fp4_dequantize if book == "fp4" else oracle.dequantize
    p, a = quant(w.reshape(-1))
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    qt = nf4._QUANT_TYPES[book]
    if scales == "plain":
        qw = nf4.QuantizedWeight(packed=dev(p), rows=experts * n, cols=k, absmax=dev(a), quant_type=qt)
    else:
        code = oracle.DQ_E4M3 if scales == "e4m3" else oracle.DQ_INT8
        q, s, m = oracle.double_quant(a, 256, code)
        a = oracle.absmax_reconstruct(q, s, m, 256, code)
        qw = nf4.QuantizedWeight(packed=dev(p), rows=experts * n, cols=k, absmax_q=dev(q), absmax_scale=dev(s),
                                 absmax_mean=torch.tensor([m], dtype=torch.float32, device="cuda"),
                                 dq_code=nf4._DQ_CODES[scales], quant_type=qt)
    bits = deq(p, a, experts * n * k, 64, "bf16")
    wc = dev(bits.view(np.int16)).view(torch.bfloat16).double().reshape(experts, n, k)
    return qw, wc


def offsets_of(counts, lead=0):
    return torch.tensor(np.concatenate([[lead], lead + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def reference(wc, x, off, gradient):
    """fp64 outputs and sums of absolute values; NaN where no expert has the row"""
    o = off.tolist()
    width = wc.shape[2] if gradient else wc.shape[1]
    ref = torch.full((x.shape[0], width), float("nan"), dtype=torch.float64, device="cuda")
    s = ref.clone()
    for e in range(wc.shape[0]):
        w = wc[e] if gradient else wc[e].t()
        ref[o[e]:o[e + 1]] = x[o[e]:o[e + 1]].double() @ w
        s[o[e]:o[e + 1]] = x[o[e]:o[e + 1]].double().abs() @ w.abs()
    return ref, s


def check(y, ref, s, terms):
    tol = ref.abs() * 2.0 ** -8 + (terms * 17 / 16 + 8) * 2.0 ** -23 * s * (1 + 2.0 ** -8)
    err = (y.double() - ref).abs()
    ok = (err <= tol) | torch.isnan(ref)
    assert bool(ok.all()), f"{int((~ok).sum())} outputs off, worst {float((err / tol).nan_to_num().max()):.2f} of tol"


def activations(m, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(m, width, generator=g, device="cuda").bfloat16()


COUNTS = [
    [1],
    [0, 1, 0],
    [3, 0, 16, 17],
    [64, 65, 1, 63],
    [5, 0, 0, 0, 0, 0, 0, 2],
    [300, 0, 7],
    [256, 257, 255, 129],
    [1000, 1],
    [0, 0, 513],
    [1] * 40,
    [2, 0] * 128,
]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
@pytest.mark.parametrize("gradient", [False, True])
def test_ragged_counts(counts, gradient):
    n, k = (192, 256) if gradient else (256, 192)
    qw, wc = make_stack(len(counts), n, k)
    off = offsets_of(counts)
    x = activations(sum(counts), n if gradient else k, 1)
    y = (nf4.gemm_experts_dx if gradient else nf4.gemm_experts)(qw, x, off, len(counts))
    check(y, *reference(wc, x, off, gradient), n if gradient else k)
    nf4.check_device_error()


@pytest.mark.parametrize("book", ["nf4", "fp4"])
@pytest.mark.parametrize("scales", ["plain", "e4m3", "int8"])
@pytest.mark.parametrize("n,k", [(128, 128), (384, 1024), (1024, 384), (2048, 1408)])
def test_weight_forms(book, scales, n, k):
    counts = [33, 0, 130]
    qw, wc = make_stack(3, n, k, book, scales)
    off = offsets_of(counts)
    x, dy = activations(163, k, 2), activations(163, n, 3)
    check(nf4.gemm_experts(qw, x, off, 3), *reference(wc, x, off, False), k)
    check(nf4.gemm_experts_dx(qw, dy, off, 3), *reference(wc, dy, off, True), n)
    nf4.check_device_error()


@pytest.mark.parametrize("n,k", [(128, 64), (640, 64), (128, 4160), (64, 128), (64, 4224), (4160, 128)])
def test_short_and_long_reductions(n, k):
    """one stage, and more stages than the rings hold"""
    qw, wc = make_stack(2, n, k)
    off = offsets_of([9, 70])
    if n % 128 == 0:
        x = activations(79, k, 4)
        check(nf4.gemm_experts(qw, x, off, 2), *reference(wc, x, off, False), k)
    if k % 128 == 0:
        dy = activations(79, n, 5)
        check(nf4.gemm_experts_dx(qw, dy, off, 2), *reference(wc, dy, off, True), n)
    nf4.check_device_error()


@pytest.mark.parametrize("out_cols", [128, 384, 640])
@pytest.mark.parametrize("red", [64, 192, 1024])
@pytest.mark.parametrize("gradient", [False, True])
def test_pairs_at_odd_widths(out_cols, red, gradient):
    """many rows per expert (CTA pairs share 256 output columns): a last column tile of 128, one or three blocks of
    reduction, tiles of 16 to 256 rows, the last expert's weight at the end of the stack"""
    counts = [257, 1, 0, 130, 512, 31]
    n, k = (red, out_cols) if gradient else (out_cols, red)
    qw, wc = make_stack(len(counts), n, k, seed=5)
    off = offsets_of(counts, lead=3)
    x = activations(sum(counts) + 5, n if gradient else k, 18)
    f = nf4.gemm_experts_dx if gradient else nf4.gemm_experts
    out = torch.full((x.shape[0], out_cols), 3.5, dtype=torch.bfloat16, device="cuda")
    f(qw, x, off, len(counts), out=out)
    check(out, *reference(wc, x, off, gradient), red)
    assert bool((out[:3] == 3.5).all()) and bool((out[-2:] == 3.5).all())
    for _ in range(3):
        assert torch.equal(f(qw, x, off, len(counts), out=out.clone()), out)
    nf4.check_device_error()


@pytest.mark.parametrize("out_cols,red", [(2176, 64), (2176, 192), (1664, 1088), (4224, 1024)])
@pytest.mark.parametrize("gradient", [False, True])
def test_pairs_on_a_full_gpu(out_cols, red, gradient):
    """enough tiles that pairs are taken: a last column tile of 128, odd reductions, ragged tiles, experts without rows"""
    counts = [257, 1, 0, 130, 512, 31, 700, 256]
    n, k = (red, out_cols) if gradient else (out_cols, red)
    qw, wc = make_stack(len(counts), n, k, seed=6)
    off = offsets_of(counts, lead=3)
    x = activations(sum(counts) + 5, n if gradient else k, 20)
    f = nf4.gemm_experts_dx if gradient else nf4.gemm_experts
    out = torch.full((x.shape[0], out_cols), 3.5, dtype=torch.bfloat16, device="cuda")
    f(qw, x, off, len(counts), out=out)
    check(out, *reference(wc, x, off, gradient), red)
    assert bool((out[:3] == 3.5).all()) and bool((out[-2:] == 3.5).all())
    for _ in range(3):
        assert torch.equal(f(qw, x, off, len(counts), out=out.clone()), out)
    nf4.check_device_error()


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("counts", [[1000, 1], [300, 300], [0, 129]])
def test_many_rows_few_tiles(gradient, counts):
    """many rows but a narrow output: tiles of one CTA, split over the reduction; a workspace too small is refused"""
    n, k = (4096, 256) if gradient else (256, 4096)
    qw, wc = make_stack(2, n, k, seed=7)
    off = offsets_of(counts)
    x = activations(sum(counts), n if gradient else k, 21)
    f = nf4.gemm_experts_dx if gradient else nf4.gemm_experts
    y = f(qw, x, off, 2)
    check(y, *reference(wc, x, off, gradient), n if gradient else k)
    for _ in range(5):
        assert torch.equal(f(qw, x, off, 2), y)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        f(qw, x, off, 2, workspace=torch.zeros(1024, dtype=torch.uint8, device="cuda"))
    nf4.check_device_error()


def test_side_stream_argument():
    """stream=: the output is allocated and written on that stream"""
    qw, wc = make_stack(2, 128, 128)
    x, off = activations(60, 128, 19), offsets_of([20, 40])
    ref = reference(wc, x, off, False)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = nf4.gemm_experts(qw, x, off, 2, stream=side)
    dx = nf4.gemm_experts_dx(qw, x, off, 2, stream=side)
    side.synchronize()
    check(y, *ref, 128)
    check(dx, *reference(wc, x, off, True), 128)


@pytest.mark.parametrize("gradient", [False, True])
def test_many_tiles_per_cta(gradient):
    """several hundred units on the grid: every CTA walks many tiles of several experts, repeated calls agree bit for bit"""
    counts = [700, 0, 31, 520, 258, 64, 1, 410]
    n = k = 2048
    qw, wc = make_stack(len(counts), n, k)
    off = offsets_of(counts)
    x = activations(sum(counts), k, 6)
    f = nf4.gemm_experts_dx if gradient else nf4.gemm_experts
    y = f(qw, x, off, len(counts))
    check(y, *reference(wc, x, off, gradient), k)
    for _ in range(5):
        assert torch.equal(f(qw, x, off, len(counts)), y)
    nf4.check_device_error()


@pytest.mark.parametrize("gradient", [False, True])
def test_rows_of_no_expert_stay(gradient):
    """rows before the first and behind the last expert keep their values, also where they hold NaN inputs"""
    qw, wc = make_stack(3, 256, 256)
    off = offsets_of([5, 0, 30], lead=7)
    x = activations(50, 256, 7)
    x[:7] = float("nan")
    x[42:] = float("inf")
    f = nf4.gemm_experts_dx if gradient else nf4.gemm_experts
    out = torch.full((50, 256), 3.5, dtype=torch.bfloat16, device="cuda")
    assert f(qw, x, off, 3, out=out) is out
    ref, s = reference(wc, x, off, gradient)
    check(out, ref, s, 256)
    assert bool((out[:7] == 3.5).all()) and bool((out[42:] == 3.5).all())
    none = torch.full((50, 256), 3.5, dtype=torch.bfloat16, device="cuda")
    f(qw, x, torch.full((4,), 20, dtype=torch.int32, device="cuda"), 3, out=none)
    assert bool((none == 3.5).all())


@pytest.mark.parametrize("gradient", [False, True])
def test_offsets_outside_the_rows_are_held(gradient):
    """offsets below 0 and above m are held to 0 and m: every row is written by its expert, nothing outside"""
    qw, wc = make_stack(2, 128, 128)
    x = activations(20, 128, 8)
    off = torch.tensor([-1000, 4, 2_000_000_000], dtype=torch.int32, device="cuda")
    f = nf4.gemm_experts_dx if gradient else nf4.gemm_experts
    buf = torch.full((28, 128), 3.5, dtype=torch.bfloat16, device="cuda")
    f(qw, x, off, 2, out=buf[4:24])
    check(buf[4:24], *reference(wc, x, offsets_of([4, 16]), gradient), 128)
    assert bool((buf[:4] == 3.5).all()) and bool((buf[24:] == 3.5).all())


@pytest.mark.parametrize("gradient", [False, True])
def test_nan_and_inf_rows_do_not_mix(gradient):
    """tiles reach into the next expert's rows; a NaN or Inf row changes no other row"""
    qw, _ = make_stack(2, 128, 128)
    off = offsets_of([10, 40])
    x = activations(50, 128, 9)
    f = nf4.gemm_experts_dx if gradient else nf4.gemm_experts
    clean = f(qw, x, off, 2)
    x[10] = float("nan")
    x[30] = float("inf")
    y = f(qw, x, off, 2)
    keep = torch.ones(50, dtype=torch.bool, device="cuda")
    keep[10] = keep[30] = False
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[10]).all())


def test_matches_the_single_weight_products():
    """one expert with every row: within tolerance of gemm and gemm_dx, on the same weight"""
    qw, wc = make_stack(1, 512, 512)
    off = offsets_of([300])
    x = activations(300, 512, 10)
    for f, g, grad in ((nf4.gemm_experts, nf4.gemm, False), (nf4.gemm_experts_dx, nf4.gemm_dx, True)):
        ref, s = reference(wc, x, off, grad)
        check(f(qw, x, off, 1), ref, s, 512)
        check(g(qw, x), ref, s, 512)


def test_one_hot_rows_return_the_weight():
    qw, wc = make_stack(2, 128, 192)
    x = torch.zeros(2 * 192, 192, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(384), torch.arange(384) % 192] = 1.0
    y = nf4.gemm_experts(qw, x, offsets_of([192, 192]), 2)
    assert torch.equal(y[:192].double(), wc[0].t()) and torch.equal(y[192:].double(), wc[1].t())
    qw, wc = make_stack(2, 192, 128)
    dy = torch.zeros(2 * 192, 192, dtype=torch.bfloat16, device="cuda")
    dy[torch.arange(384), torch.arange(384) % 192] = 1.0
    dx = nf4.gemm_experts_dx(qw, dy, offsets_of([192, 192]), 2)
    assert torch.equal(dx[:192].double(), wc[0]) and torch.equal(dx[192:].double(), wc[1])


def test_graph_replay_reads_the_offsets_anew():
    """a captured call follows the offsets and rows that lie in its buffers at each replay"""
    qw, wc = make_stack(4, 256, 256)
    x = activations(96, 256, 11)
    off = offsets_of([24, 24, 24, 24])
    y, dx = (torch.zeros(96, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wf, wb = (torch.zeros(max(16, f(qw, 4, 96)), dtype=torch.uint8, device="cuda")
              for f in (nf4.gemm_experts_workspace_bytes, nf4.gemm_experts_dx_workspace_bytes))
    nf4.gemm_experts(qw, x, off, 4, out=y, workspace=wf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nf4.gemm_experts(qw, x, off, 4, out=y, workspace=wf)
        nf4.gemm_experts_dx(qw, y, off, 4, out=dx, workspace=wb)
    for counts in ([96, 0, 0, 0], [0, 1, 94, 1], [30, 31, 32, 3]):
        off.copy_(offsets_of(counts))
        x.copy_(activations(96, 256, sum(counts[:2])))
        graph.replay()
        torch.cuda.synchronize()
        check(y, *reference(wc, x, off, False), 256)
        check(dx, *reference(wc, y, off, True), 256)
    nf4.check_device_error()


def test_two_streams_at_once():
    """calls on two streams, each with its own workspace and outputs, run beside one another"""
    qw, wc = make_stack(4, 1024, 1024)
    offs = [offsets_of([1, 30, 0, 9]), offsets_of([0, 2, 300, 5])]
    xs = [activations(40, 1024, 12), activations(307, 1024, 13)]
    refs = [reference(wc, x, o, False) for x, o in zip(xs, offs)]
    want = [nf4.gemm_experts(qw, x, o, 4) for x, o in zip(xs, offs)]
    wss = [torch.zeros(max(16, nf4.gemm_experts_workspace_bytes(qw, 4, x.shape[0])), dtype=torch.uint8,
                       device="cuda") for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(nf4.gemm_experts(qw, xs[i], offs[i], 4, workspace=wss[i]))
    torch.cuda.synchronize()
    for i in range(2):
        check(outs[i][0], *refs[i], 1024)
        for o in outs[i]:
            assert torch.equal(o, want[i])
    nf4.check_device_error()


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("counts", [[1, 0, 0, 0], [0, 1, 0, 1], [2, 2, 2, 2], [0, 64, 3, 0], [33, 0, 0, 40]])
def test_few_units_split_the_reduction(gradient, counts):
    """single tokens: fewer units than SMs, the reduction split over CTAs; one workspace for calls in a row, equal bits"""
    n, k = (4096, 1024) if gradient else (1024, 4096 + 64)
    qw, wc = make_stack(4, n, k)
    off = offsets_of(counts)
    f, size = ((nf4.gemm_experts_dx, nf4.gemm_experts_dx_workspace_bytes) if gradient else
               (nf4.gemm_experts, nf4.gemm_experts_workspace_bytes))
    x = activations(sum(counts), n if gradient else k, 17)
    need = size(qw, 4, sum(counts))
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    y = f(qw, x, off, 4, workspace=ws)
    check(y, *reference(wc, x, off, gradient), n if gradient else k)
    for _ in range(10):
        assert torch.equal(f(qw, x, off, 4, workspace=ws), y)
    other = offsets_of(counts[::-1])
    check(f(qw, x, other, 4, workspace=ws), *reference(wc, x, other, gradient), n if gradient else k)
    assert torch.equal(f(qw, x, off, 4), y)  # a workspace of its own
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        f(qw, x, off, 4, workspace=ws[:need - 16])
    nf4.check_device_error()


def moe_forward(up, down, experts, x, off):
    """h = silu(gate) * value of the stacked [gate | value] rows, then the down projections; all rows sorted"""
    h = nf4.gemm_experts(up, x, off, experts).float()
    g, v = h.chunk(2, 1)
    act = (torch.nn.functional.silu(g) * v).bfloat16()
    return h, act, nf4.gemm_experts(down, act, off, experts)


def test_mixture_of_experts_block():
    """a routed block built of the library's calls: rows sorted by a router's choice, up, gate, down, and the gradient
    back to the rows; each step against fp64, the gradient also against differences of the fp64 block"""
    experts, d, f, tokens = 4, 256, 384, 120
    up, wu = make_stack(experts, 2 * f, d, seed=1)
    down, wd = make_stack(experts, d, f, seed=2)
    logits = torch.randn(tokens, experts, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    choice = logits.topk(2).indices.reshape(-1)
    order = torch.argsort(choice, stable=True)
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(choice, minlength=experts).cumsum(0)
    rows = activations(tokens, d, 14)[order // 2].contiguous()
    h, act, y = moe_forward(up, down, experts, rows, off)
    check(h.bfloat16(), *reference(wu, rows, off, False), d)
    check(y, *reference(wd, act, off, False), f)
    # backward: dy -> d act -> d [gate | value] -> d rows
    dy = activations(2 * tokens, d, 15)
    dact = nf4.gemm_experts_dx(down, dy, off, experts)
    check(dact, *reference(wd, dy, off, True), d)
    g, v = h.chunk(2, 1)
    sg = torch.sigmoid(g)
    da = dact.float()
    dh = torch.cat([da * v * (sg + g * sg * (1 - sg)), da * g * sg], 1).bfloat16()
    dx = nf4.gemm_experts_dx(up, dh, off, experts)
    check(dx, *reference(wu, dh, off, True), 2 * f)

    def block(r):  # the block in fp64, no 16-bit roundings in between
        o = off.tolist()
        out = []
        for e in range(experts):
            hh = r[o[e]:o[e + 1]] @ wu[e].t()
            out.append((torch.nn.functional.silu(hh[:, :f]) * hh[:, f:]) @ wd[e].t())
        return torch.cat(out)

    r64 = rows.double()
    u = torch.randn(r64.shape, device="cuda", dtype=torch.float64, generator=torch.Generator(device="cuda").manual_seed(4))
    eps = 1e-5
    slope = ((block(r64 + eps * u) - block(r64 - eps * u)) * dy.double()).sum(1) / (2 * eps)
    got = (dx.double() * u).sum(1)
    # three bf16 roundings lie between (dact, dh, dx), each at most 2^-8 of its value, and the product's own of h and
    # act: together below 5 * 2^-8 of the sum of the terms' sizes along the row
    scale = (dx.double().abs() * u.abs()).sum(1) + \
        torch.cat([(dh.double().abs()[a:b] @ wu[e].abs()) for e, (a, b) in
                   enumerate(zip(off.tolist()[:-1], off.tolist()[1:]))]).mul(u.abs()).sum(1)
    assert bool(((slope - got).abs() <= 5 * 2.0 ** -8 * scale).all())
    # combine: the two experts' rows of a token, back in the tokens' order
    back = torch.empty_like(y)
    back[order] = y
    ref = torch.empty(2 * tokens, d, dtype=torch.float64, device="cuda")
    ref[order] = reference(wd, act, off, False)[0]
    assert torch.allclose(back.reshape(tokens, 2, d).double().sum(1), ref.reshape(tokens, 2, d).sum(1), rtol=0.02, atol=0.02)


def test_experts_refusals():
    qw, _ = make_stack(2, 128, 128)
    x, off = activations(10, 128, 16), offsets_of([5, 5])
    for f in (nf4.gemm_experts, nf4.gemm_experts_dx):
        with pytest.raises(ValueError):
            f(qw, x, off.long(), 2)
        with pytest.raises(ValueError):
            f(qw, x, off, 3)
        with pytest.raises(ValueError):
            f(qw, x[:, :64].contiguous(), off, 2)
        with pytest.raises(ValueError):
            f(qw, x.t(), off, 2)
        with pytest.raises(ValueError):
            f(qw, x, off.cpu(), 2)
        with pytest.raises(TypeError):
            f(qw, x.float(), off, 2)
        with pytest.raises(ValueError):
            f(qw, x, off, 2, out=torch.zeros(10, 64, dtype=torch.bfloat16, device="cuda"))
        assert f(qw, x[:0], torch.zeros(3, dtype=torch.int32, device="cuda"), 2).shape == (0, 128)
    odd = nf4.QuantizedWeight(packed=qw.packed, rows=256, cols=128, absmax=torch.zeros(512, device="cuda"),
                              blocksize=128)
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        nf4.gemm_experts(odd, x, off, 2)
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):  # 64 rows per expert are no 128-row tile
        nf4.gemm_experts(qw, x, torch.zeros(5, dtype=torch.int32, device="cuda"), 4)
