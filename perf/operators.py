"""Cases, plain forms and 64-bit definitions of the products with 4-bit weights that perf measurements run.

Operators:
  gemv_groups        y[b, n] = sum_g s[n, g] sum_{k in g} (q[n, k] - z[n, g]) x[b, k]: the decode product with weights
                     of 4 bits, one 16-bit scale (and one zero point of 0..15, or 8 for all) per group of 32, 64 or
                     128 columns; x bf16 or fp16, 1 to 8 rows.
  round_trip_groups  quantize_groups then dequantize_groups: the codes, scales and zero points of a weight, and the
                     values they stand for.
  gemm_experts       y[t] = Wc_e(t) x[t]: rows sorted by expert (offsets on the GPU), each multiplied by its expert's
                     NF4 or FP4 weight, Wc = bf16(code * scale) as in the library's other products.
  gemm_experts_dx    dx[t] = dy[t] Wc_e(t): the input gradient of gemm_experts through the frozen weights.

`run` with `own` false is the plain form (elementary torch operations in fp32, one rounding at the end); with `own`
true it makes the library's calls.  `exact` is the definition in fp64, written apart from the plain form.
"""
import math
import random
import statistics

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 64       # NF4 / FP4 level-1 block
DQ_BLOCK = 256   # absmax values per second-level scale
WEIGHT_STD = 0.02
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through a key/value projection of an 8B decoder layer: the smallest call, latency counts
        {"name": "gemv_groups_1024x4096_b1", "op": "gemv_groups", "rows": 1024, "cols": 4096, "group": 128, "batch": 1,
         "zeros": True, "type": "bf16"},
        # one token through the down projection: a long reduction
        {"name": "gemv_groups_4096x14336_b1_f16", "op": "gemv_groups", "rows": 4096, "cols": 14336, "group": 128,
         "batch": 1, "zeros": False, "type": "f16"},
        # eight sequences decoded together through the gate projection, finer groups
        {"name": "gemv_groups_14336x4096_b8_g64", "op": "gemv_groups", "rows": 14336, "cols": 4096, "group": 64,
         "batch": 8, "zeros": True, "type": "bf16"},
        # an output layer with an odd number of rows, a reduction that no power of two divides, the finest groups
        {"name": "gemv_groups_32003x4128_b3_g32", "op": "gemv_groups", "rows": 32003, "cols": 4128, "group": 32,
         "batch": 3, "zeros": True, "type": "bf16"},
        # a projection quantized as a model loads, expanded again for a long prompt
        {"name": "round_trip_4096x4096_bf16", "op": "round_trip_groups", "rows": 4096, "cols": 4096, "group": 128,
         "zeros": True, "src": "bf16", "type": "bf16"},
        # the same for an fp32 master weight with symmetric groups and an odd number of rows
        {"name": "round_trip_14337x4096_f32", "op": "round_trip_groups", "rows": 14337, "cols": 4096, "group": 64,
         "zeros": False, "src": "f32", "type": "f16"},
        # 8 sequences decoded, two experts of eight each: 16 rows, some experts without any
        {"name": "experts_8x14336x4096_t16", "op": "gemm_experts", "experts": 8, "rows": 14336, "cols": 4096,
         "tokens": 16, "route": 1, "skew": 1.0, "double_quant": True, "book": "nf4"},
        # many narrow experts, a few hundred rows, plain fp32 scales
        {"name": "experts_64x1024x2048_t777", "op": "gemm_experts", "experts": 64, "rows": 1024, "cols": 2048,
         "tokens": 777, "route": 2, "skew": 1.0, "double_quant": False, "book": "nf4"},
        # a prompt of 2048 tokens, two experts each: ragged large products
        {"name": "experts_8x14336x4096_t4096", "op": "gemm_experts", "experts": 8, "rows": 14336, "cols": 4096,
         "tokens": 4096, "route": 3, "skew": 0.5, "double_quant": True, "book": "nf4"},
        # a short training sequence through the down projections' experts, back to their input
        {"name": "experts_dx_16x2048x1024_t300", "op": "gemm_experts_dx", "experts": 16, "rows": 2048, "cols": 1024,
         "tokens": 300, "route": 4, "skew": 1.0, "double_quant": True, "book": "nf4"},
        # the gradient of the 4096-row product
        {"name": "experts_dx_8x14336x4096_t4096", "op": "gemm_experts_dx", "experts": 8, "rows": 14336, "cols": 4096,
         "tokens": 4096, "route": 3, "skew": 0.5, "double_quant": True, "book": "nf4"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv_groups", "gemv_groups", "round_trip_groups", "gemm_experts", "gemm_experts",
                     "gemm_experts_dx"])
    if op == "gemv_groups":
        group = rng.choice([32, 64, 128])
        while True:
            rows, cols = _log(rng, 64, 32768), group * max(1, _log(rng, 256, 16384) // group)
            if 1 << 16 <= rows * cols <= 14336 * 4096:
                break
        return {"op": op, "rows": rows, "cols": cols, "group": group, "batch": rng.randint(1, 8),
                "zeros": rng.random() < 0.5, "type": rng.choice(["bf16", "f16"])}
    if op == "round_trip_groups":
        group = rng.choice([32, 64, 128])
        while True:
            rows, cols = _log(rng, 64, 16384), group * max(1, _log(rng, 256, 16384) // group)
            if 1 << 18 <= rows * cols <= 14336 * 4096:
                break
        return {"op": op, "rows": rows, "cols": cols, "group": group, "zeros": rng.random() < 0.5,
                "src": rng.choice(["f32", "bf16", "f16"]), "type": rng.choice(["bf16", "f16"])}
    experts = _log(rng, 2, 64)
    while True:
        rows, cols = 128 * _log(rng, 2, 112), 128 * _log(rng, 2, 112)
        if experts * rows * cols <= 8 * 14336 * 4096 and rows * cols >= 1 << 18:
            break
    while True:
        tokens = _log(rng, 1, 8192)
        if tokens * rows * cols <= 4096 * 14336 * 4096:
            break
    return {"op": op, "experts": experts, "rows": rows, "cols": cols, "tokens": tokens,
            "route": rng.randrange(1 << 30), "skew": rng.choice([0.0, 0.5, 1.0]),
            "double_quant": rng.random() < 0.7, "book": rng.choice(["nf4", "nf4", "fp4"])}


def _counts(case):
    """rows per expert: each row picks an expert, expert i with weight (i + 1)^-skew.  The numbers belong to the
    case; which expert gets which of them goes by the seed."""
    rng = random.Random(case["route"])
    e = case["experts"]
    picks = rng.choices(range(e), weights=[(i + 1.0) ** -case["skew"] for i in range(e)], k=case["tokens"])
    counts = [0] * e
    for p in picks:
        counts[p] += 1
    return counts


def work(case):
    op = case["op"]
    if op in ("gemv_groups", "round_trip_groups"):
        n, k, g = case["rows"], case["cols"], case["group"]
        meta = n * (k // g) * (3 if case["zeros"] else 2)  # 16-bit scale, 8-bit zero point
        if op == "gemv_groups":
            return {"bytes": n * k // 2 + meta + 2 * case["batch"] * (n + k), "flops": 2 * case["batch"] * n * k}
        # the weight in; codes, scales and zero points out and in again; the values out
        size = 4 if case["src"] == "f32" else 2
        return {"bytes": n * k * (size + 2) + 2 * (n * k // 2 + meta), "flops": 4 * n * k}
    n, k, t = case["rows"], case["cols"], case["tokens"]
    active = sum(1 for c in _counts(case) if c > 0)
    weights = n * k
    scales = n * k // BLOCK * (1 if case["double_quant"] else 4)
    if case["double_quant"]:
        scales += 4 * (n * k // BLOCK // DQ_BLOCK)
    return {"bytes": active * (weights // 2 + scales) + 2 * t * (n + k), "flops": 2 * t * n * k}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _nf4_levels():
    """16 normal quantiles scaled to [-1, 1], in fp32"""
    nd = statistics.NormalDist()
    p = 0.5 * ((1 - 1 / 30) + (1 - 1 / 32))
    v = ([-nd.inv_cdf(0.5 + (p - 0.5) * (k / 7)) for k in range(7, 0, -1)] + [0.0] +
         [nd.inv_cdf(0.5 + (p - 0.5) * (k / 8)) for k in range(1, 9)])
    top = max(abs(a) for a in v)
    return torch.tensor([a / top for a in v], dtype=torch.float64).float()


def _fp4_levels():
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64) / 6
    return torch.cat([mag, -mag]).float()


def _levels(book):
    return (_nf4_levels() if book == "nf4" else _fp4_levels()).to(DEV)


def _pack_pairs(codes):
    """two codes a byte, the first in the high nibble"""
    return (codes[:, 0::2] << 4) | codes[:, 1::2]


def _block_weight(case, g):
    """A stack of experts' weights [experts * rows, cols] as they lie in memory after loading: normal weights in blocks
    of 64, each code the nearest level of w / absmax; the absmax array in fp32, or with its mean removed and coded as
    E4M3 in blocks of 256."""
    n, k = case["rows"], case["cols"]
    lv = _levels(case["book"])
    order = torch.argsort(lv)
    mid = (lv[order][1:] + lv[order][:-1]) / 2
    packed, absmax = [], []
    for _ in range(case["experts"]):
        w = torch.randn((n * k // BLOCK, BLOCK), generator=g, device=DEV) * WEIGHT_STD
        a = w.abs().amax(1)
        idx = order[torch.bucketize(w / a[:, None], mid, out_int32=True)].to(torch.uint8)
        packed.append(_pack_pairs(idx).reshape(-1))
        absmax.append(a)
        del w, idx
    out = {"packed": torch.cat(packed), "absmax": None}
    a = torch.cat(absmax)
    if not case["double_quant"]:
        out["absmax"] = a
        return out
    mean = (a.double().mean()).float().reshape(1)
    r = a - mean
    pad = -r.numel() % DQ_BLOCK
    rb = torch.nn.functional.pad(r, (0, pad)).reshape(-1, DQ_BLOCK)
    m = rb.abs().amax(1)
    q = (rb / m[:, None].clamp_min(1e-30) * 448.0).to(torch.float8_e4m3fn).reshape(-1)[: r.numel()]
    out.update(q=q.contiguous().view(torch.uint8), scale=m, mean=mean)
    return out


def _group_codes(case, w):
    """codes [rows, cols] 0..15, scales [rows, groups], zero points [rows, groups] or None: the groups' scale is their
    range / 15 (with zeros) or their absmax / 7, rounded to the scales' type, and w / scale goes to the nearest code"""
    n, k, g = case["rows"], case["cols"], case["group"]
    wg = w.float().reshape(n, k // g, g)
    const = lambda v: torch.full((), v, device=DEV)  # noqa: E731  (a tensor: a division, not a product with 1 / v)
    if case["zeros"]:
        lo, hi = wg.amin(2).clamp_max(0), wg.amax(2).clamp_min(0)
        s = ((hi - lo) / const(15.0)).to(TYPES[case["type"]])
        sf = s.float()
        safe = torch.where(sf == 0, torch.ones_like(sf), sf)
        z = torch.round(-lo / safe).clamp(0, 15)
        z = torch.where(sf == 0, torch.zeros_like(z), z)
    else:
        s = (wg.abs().amax(2) / const(7.0)).to(TYPES[case["type"]])
        sf = s.float()
        safe = torch.where(sf == 0, torch.ones_like(sf), sf)
        z = torch.full_like(sf, 8.0)
    c = torch.round(wg / safe[..., None]) + z[..., None]
    c = torch.where(sf[..., None] == 0, z[..., None], c.clamp(0, 15))
    return c.to(torch.uint8).reshape(n, k), s, z.to(torch.uint8) if case["zeros"] else None


def _pack_groups(codes):
    """eight codes a little-endian 32-bit word: code j in nibble j / 2 of the low half (j even) or the high half (j
    odd), as the library's group weights keep them"""
    n, k = codes.shape
    c = codes.reshape(n, k // 8, 8)
    b = [c[..., 0] | (c[..., 2] << 4), c[..., 4] | (c[..., 6] << 4), c[..., 1] | (c[..., 3] << 4),
         c[..., 5] | (c[..., 7] << 4)]
    return torch.stack(b, -1).reshape(n, k // 2)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    op = case["op"]
    if op == "round_trip_groups":
        st["w"] = _normal((case["rows"], case["cols"]), g, WEIGHT_STD, TYPES[case["src"]])
        return st
    if op == "gemv_groups":
        w = _normal((case["rows"], case["cols"]), g, WEIGHT_STD, torch.float32)
        codes, st["scale"], st["zero"] = _group_codes(case, w)
        st["packed"] = _pack_groups(codes)
        st["x"] = _normal((case["batch"], case["cols"]), g, 1.0, TYPES[case["type"]])
        if own:
            import qlora_block_absmax_b200 as nf4
            st["weight"] = nf4.GroupWeight(packed=st["packed"], scale=st["scale"], zero=st["zero"], rows=case["rows"],
                                           cols=case["cols"], group=case["group"])
        return st
    st.update(_block_weight(case, g))
    counts = _counts(case)
    random.Random(seed).shuffle(counts)
    st["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    width = case["cols"] if op == "gemm_experts" else case["rows"]
    st["x"] = _normal((case["tokens"], width), g, 1.0, torch.bfloat16)
    if own:
        import qlora_block_absmax_b200 as nf4
        e = case["experts"]
        qt = nf4._QUANT_TYPES[case["book"]]
        if case["double_quant"]:
            qw = nf4.QuantizedWeight(packed=st["packed"], rows=e * case["rows"], cols=case["cols"], absmax_q=st["q"],
                                     absmax_scale=st["scale"], absmax_mean=st["mean"], quant_type=qt)
        else:
            qw = nf4.QuantizedWeight(packed=st["packed"], rows=e * case["rows"], cols=case["cols"],
                                     absmax=st["absmax"], quant_type=qt)
        st["weight"] = qw
        size = nf4.gemm_experts_workspace_bytes if op == "gemm_experts" else nf4.gemm_experts_dx_workspace_bytes
        st["workspace"] = torch.zeros(max(16, size(qw, e, case["tokens"])), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        import qlora_block_absmax_b200 as nf4
        op = case["op"]
        if op == "gemv_groups":
            return nf4.gemv_groups(st["weight"], st["x"])
        if op == "round_trip_groups":
            gw = nf4.quantize_groups(st["w"], group=case["group"], symmetric=not case["zeros"],
                                     scale_dtype=TYPES[case["type"]])
            vals = nf4.dequantize_groups(gw, TYPES[case["type"]])
            return [vals, gw.scale, gw.zero] if case["zeros"] else [vals, gw.scale]
        f = nf4.gemm_experts if op == "gemm_experts" else nf4.gemm_experts_dx
        return f(st["weight"], st["x"], st["offsets"], case["experts"], workspace=st["workspace"])
    return _PLAIN[case["op"]](case, st)


def _plain_gemv(case, st):
    n, k, g = case["rows"], case["cols"], case["group"]
    b = st["packed"].reshape(n, k // 8, 4)
    lo, hi = b & 15, b >> 4
    codes = torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1],
                         hi[..., 3]], -1).reshape(n, k // g, g)
    z = st["zero"].float()[..., None] if case["zeros"] else 8.0
    w = ((codes.float() - z) * st["scale"].float()[..., None]).reshape(n, k)
    return (st["x"].float() @ w.t()).to(st["x"].dtype)


def _plain_round_trip(case, st):
    codes, s, z = _group_codes(case, st["w"])
    n, k, g = case["rows"], case["cols"], case["group"]
    zf = z.float()[..., None] if case["zeros"] else 8.0
    vals = (codes.reshape(n, k // g, g).float() - zf) * s.float()[..., None]
    vals = vals.reshape(n, k).to(TYPES[case["type"]])
    return [vals, s, z] if case["zeros"] else [vals, s]


def _plain_scales(case, st):
    """fp32 scale of every level-1 block"""
    if not case["double_quant"]:
        return st["absmax"]
    unit = st["q"].view(torch.float8_e4m3fn).float() / torch.full((), 448.0, device=DEV)
    return unit * st["scale"].repeat_interleave(DQ_BLOCK)[: unit.numel()] + st["mean"]


def _plain_expert_weight(case, st, a, lv, e):
    """expert e's weight as the products use it, bf16 values in fp32 [rows, cols]"""
    n, k = case["rows"], case["cols"]
    p = st["packed"][e * n * k // 2:(e + 1) * n * k // 2].int()
    codes = torch.stack([p >> 4, p & 15], -1).reshape(-1, BLOCK)
    w = lv[codes] * a[e * n * k // BLOCK:(e + 1) * n * k // BLOCK, None]
    return w.bfloat16().float().reshape(n, k)


def _plain_experts(case, st):
    back = case["op"] == "gemm_experts_dx"
    x = st["x"].float()
    y = torch.empty((case["tokens"], case["cols" if back else "rows"]), dtype=torch.bfloat16, device=DEV)
    a, lv = _plain_scales(case, st), _levels(case["book"])
    off = st["offsets"].tolist()
    for e in range(case["experts"]):
        if off[e + 1] > off[e]:
            w = _plain_expert_weight(case, st, a, lv, e)
            xe = x[off[e]:off[e + 1]]
            y[off[e]:off[e + 1]] = (xe @ (w if back else w.t())).bfloat16()
    return y


_PLAIN = {"gemv_groups": _plain_gemv, "round_trip_groups": _plain_round_trip, "gemm_experts": _plain_experts,
          "gemm_experts_dx": _plain_experts}


# ------------------------------------------------------------------ the definition in 64 bits

def _round_to(v, dtype):
    """fp64 values rounded to fp32 and then to `dtype`, back in fp64"""
    return v.float().to(dtype).double()


def _exact_groups(w, n, k, g, zeros, dtype):
    """codes, scales and zero points of a weight in fp64.  Each step that the definition takes in fp32 is taken in fp64
    and rounded once: sums and quotients of fp32 numbers come out as if computed directly in fp32."""
    v = w.double().view(n, k // g, g)
    if zeros:
        lo = torch.minimum(v.min(2).values, v.new_zeros(()))
        hi = torch.maximum(v.max(2).values, v.new_zeros(()))
        step = _round_to((hi - lo).float().double() / v.new_full((), 15), dtype)
    else:
        step = _round_to(v.abs().max(2).values / v.new_full((), 7), dtype)
    some = step > 0
    div = torch.where(some, step, step.new_ones(()))
    if zeros:
        z = torch.where(some, (-lo / div).float().double().round().clamp(0, 15), step.new_zeros(()))
    else:
        z = torch.full_like(step, 8)
    c = ((v / div.unsqueeze(2)).float().double().round() + z.unsqueeze(2)).clamp(0, 15)
    return torch.where(some.unsqueeze(2), c, z.unsqueeze(2).expand_as(c)), step, z


def _exact_levels(book):
    if book == "fp4":
        out = []
        for bits in range(16):
            e, m = bits >> 1 & 3, bits & 1
            mag = (m * 0.5 if e == 0 else (1 + m * 0.5) * 2.0 ** (e - 1)) / 6
            out.append(-mag if bits >> 3 else mag)
        return [float(np.float32(v)) for v in out]

    def quantile(p):  # bisection on the normal tail
        lo, hi = 0.0, 8.0
        for _ in range(200):
            m = (lo + hi) / 2
            lo, hi = (m, hi) if 0.5 * math.erfc(m / math.sqrt(2)) > 1 - p else (lo, m)
        return (lo + hi) / 2

    top = (29 / 30 + 31 / 32) / 2
    q = lambda i, parts: quantile(0.5 + (top - 0.5) * i / parts) / quantile(top)  # noqa: E731
    return ([float(np.float32(-q(i, 7))) for i in range(7, 0, -1)] + [0.0] +
            [float(np.float32(q(i, 8))) for i in range(1, 9)])


def _exact_e4m3():
    out = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(-v if b >> 7 else v)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    n, k = case["rows"], case["cols"]
    if case["op"] == "round_trip_groups":
        c, s, z = _exact_groups(st["w"], n, k, case["group"], case["zeros"], TYPES[case["type"]])
        vals = ((c - z.unsqueeze(2)) * s.unsqueeze(2)).view(n, k)
        return [vals, s, z.to(torch.uint8)] if case["zeros"] else [vals, s]
    if case["op"] == "gemv_groups":
        word = st["packed"].view(torch.int32).to(torch.int64) & 0xFFFFFFFF
        c = torch.empty((n, k // 8, 8), dtype=torch.float64, device=DEV)
        for j in range(8):
            c[:, :, j] = ((word >> (4 * (j // 2) + 16 * (j % 2))) & 15).double()
        c = c.view(n, k // case["group"], case["group"])
        c -= st["zero"].double().unsqueeze(2) if case["zeros"] else 8
        c *= st["scale"].double().unsqueeze(2)
        return torch.einsum("bk,nk->bn", st["x"].double(), c.view(n, k))
    levels = torch.tensor(_exact_levels(case["book"]), dtype=torch.float64, device=DEV)
    table = torch.tensor(_exact_e4m3(), dtype=torch.float64, device=DEV)
    back = case["op"] == "gemm_experts_dx"
    y = torch.zeros((case["tokens"], k if back else n), dtype=torch.float64, device=DEV)
    off = st["offsets"].cpu().numpy()
    blocks = n * k // BLOCK
    for e in range(case["experts"]):
        if off[e] == off[e + 1]:
            continue
        b = torch.arange(e * blocks, (e + 1) * blocks, device=DEV)
        if case["double_quant"]:
            unit = (table[st["q"][b].long()] / levels.new_full((), 448)).float().double()
            prod = (unit * st["scale"].double()[b // DQ_BLOCK]).float().double()
            a = (prod + st["mean"].double()).float().double()
        else:
            a = st["absmax"].double()[b]
        bytes_ = st["packed"].view(-1, BLOCK // 2)[e * blocks:(e + 1) * blocks].long()
        w = torch.empty((blocks, BLOCK), dtype=torch.float64, device=DEV)
        w[:, 0::2] = levels[bytes_ // 16]
        w[:, 1::2] = levels[bytes_ % 16]
        w = _round_to(w * a.unsqueeze(1), torch.bfloat16).view(n, k)
        xe = st["x"][off[e]:off[e + 1]].double()
        y[off[e]:off[e + 1]] = xe.matmul(w) if back else torch.einsum("tk,nk->tn", xe, w)
    return y
