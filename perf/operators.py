"""What is measured of the MXFP4 operators: microscaled 4-bit quantisation (E2M1 elements, one
E8M0 scale per 32), the products of such operands, and the same grouped by expert.

``run`` computes each operator in plain torch (``own`` false: float32 throughout, rounded once
at the end) or through the library (``own`` true).  ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

BLOCK = 32       # elements per scale
PAD = 128        # the copies' K extent is padded to a multiple of this with zero codes
FLOOR, CEIL = 0, 1


# ---------------------------------------------------------------------------- cases
def listed():
    """kind: quantize (values of the copies), linear (serving forward with packed weights),
    train (linear layer forward and both gradients), experts / experts_train (the same with
    rows grouped by expert)."""
    return [
        # activations of one decode step of a small batch, quantised for the next product
        {"name": "quantize_decode", "kind": "quantize", "rows": 16, "cols": 4096, "dtype": "bf16",
         "col": False, "rule": FLOOR, "groups": 0, "busy": 0, "pad": 0},
        # activations of a training step: rowwise copy for the forward, columnwise for the
        # weight gradient
        {"name": "quantize_train", "kind": "quantize", "rows": 8192, "cols": 9216, "dtype": "bf16",
         "col": True, "rule": CEIL, "groups": 0, "busy": 0, "pad": 0},
        # float32 view into a wider buffer, no extent a multiple of anything
        {"name": "quantize_odd", "kind": "quantize", "rows": 4093, "cols": 1531, "dtype": "f32",
         "col": True, "rule": FLOOR, "groups": 0, "busy": 0, "pad": 5},
        # tokens sorted by expert: columnwise blocks end where an expert's rows end
        {"name": "quantize_experts", "kind": "quantize", "rows": 12001, "cols": 2048, "dtype": "bf16",
         "col": True, "rule": CEIL, "groups": 64, "busy": 57, "pad": 0},
        # one token through a linear layer
        {"name": "linear_token", "kind": "linear", "rows": 1, "cols": 4096, "out": 6144,
         "dtype": "bf16", "rule": FLOOR},
        # a batch of decoding sequences, odd sizes
        {"name": "linear_batch", "kind": "linear", "rows": 77, "cols": 2056, "out": 4999,
         "dtype": "bf16", "rule": FLOOR},
        # a prompt of 8192 tokens through the largest layer
        {"name": "linear_prompt", "kind": "linear", "rows": 8192, "cols": 6144, "out": 9216,
         "dtype": "bf16", "rule": FLOOR},
        # one training step of a linear layer: Y, dX, dW
        {"name": "train_layer", "kind": "train", "rows": 8192, "cols": 4096, "out": 6144,
         "dtype": "bf16", "rule": CEIL},
        # a small float32 layer of odd sizes
        {"name": "train_odd", "kind": "train", "rows": 1000, "cols": 777, "out": 1301,
         "dtype": "f32", "rule": CEIL},
        # a few decoding tokens, each routed to some of the experts
        {"name": "experts_decode", "kind": "experts", "rows": 24, "cols": 2048, "out": 4096,
         "dtype": "bf16", "rule": FLOOR, "groups": 32, "busy": 17},
        # a prompt's routed tokens, skewed over the experts, some without any
        {"name": "experts_prompt", "kind": "experts", "rows": 16384, "cols": 2048, "out": 4096,
         "dtype": "bf16", "rule": FLOOR, "groups": 32, "busy": 29},
        # one training step of an expert layer: Y, dX, dW of every expert
        {"name": "experts_train", "kind": "experts_train", "rows": 8191, "cols": 2048, "out": 1536,
         "dtype": "bf16", "rule": CEIL, "groups": 16, "busy": 15},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def extent(lo, hi):   # ordinary extents are multiples of 64, some are odd
        n = size(lo, hi)
        return n if rng.random() < 0.35 else max(64, n // 64 * 64)

    kind = rng.choice(["quantize", "linear", "train", "experts", "experts_train"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    rule = rng.choice([FLOOR, CEIL])
    if kind == "quantize":
        groups = rng.choice([0, 0, size(2, 64)])
        c = {"kind": kind, "rows": size(1, 8192), "cols": extent(64, 9216), "dtype": dtype,
             "col": groups > 0 or rng.random() < 0.6, "rule": rule, "groups": groups,
             "busy": max(1, groups - rng.randrange(0, 4)) if groups else 0,
             "pad": rng.choice([0, 0, 0, 3, 64])}
        return c
    c = {"kind": kind, "rows": size(1, 8192), "cols": extent(256, 6144), "out": extent(256, 6144),
         "dtype": dtype, "rule": rule}
    if kind in ("train", "experts_train"):
        c["rows"] = size(64, 8192)
        c["cols"], c["out"] = min(c["cols"], 4096), min(c["out"], 4096)
    if kind in ("experts", "experts_train"):
        c["cols"], c["out"] = min(c["cols"], 2048), min(c["out"], 4096)
        c["groups"] = size(2, 32 if kind == "experts" else 16)
        c["busy"] = max(1, c["groups"] - rng.randrange(0, 4))
    return c


def _counts(rows, groups, busy):
    """Rows of each expert before they are shuffled: shares falling as 1 / sqrt(rank) over the
    `busy` first experts, none for the others."""
    share = [1 / math.sqrt(i + 1) for i in range(busy)]
    total, counts, given = sum(share), [], 0
    run_up = 0.0
    for s in share:
        run_up += s
        upto = round(rows * run_up / total)
        counts.append(upto - given)
        given = upto
    return counts + [0] * (groups - busy)


# ---------------------------------------------------------------------------- inputs
_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _activations(n, k, dtype, gen, pad=0):
    """N(0, 1) with eight channels 30 times as large, as a view of rows `pad` elements wider."""
    x = torch.randn(n, k + pad, generator=gen, device="cuda")
    x[:, torch.randint(0, k, (8,), generator=gen, device="cuda")] *= 30
    return x.to(dtype)[:, :k]


def _gradients(n, k, dtype, gen):
    """Heavy tails: Student's t with three degrees of freedom, scaled by 1e-3."""
    z = torch.randn(n, k, generator=gen, device="cuda")
    chi = torch.zeros(n, k, device="cuda")
    for _ in range(3):
        chi += torch.randn(n, k, generator=gen, device="cuda").square_()
    return (1e-3 * z / (chi / 3).sqrt_()).to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, kind = _DTYPE[case["dtype"]], case["kind"]
    s = {"x": _activations(case["rows"], case["cols"], dtype, gen, case.get("pad", 0))}
    groups = case.get("groups", 0)
    if groups:
        order = torch.randperm(groups, generator=torch.Generator().manual_seed(int(seed))).tolist()
        counts = _counts(case["rows"], groups, case["busy"])
        counts = [counts[i] for i in order]
        s["most"] = max(counts)
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    if kind != "quantize":
        shape = (groups, case["out"], case["cols"]) if groups else (case["out"], case["cols"])
        s["w"] = (0.02 * torch.randn(shape, generator=gen, device="cuda")).to(dtype)
    if kind in ("train", "experts_train"):
        s["dy"] = _gradients(case["rows"], case["out"], dtype, gen)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    if case["kind"] in ("linear", "experts"):   # weights are held packed, as a server keeps them
        s["w_codes"], s["w_scales"] = _pack(s.pop("w"))
    return s


# ---------------------------------------------------------------------------- plain form
def _scale(amax, rule):
    """The E8M0 code of each block's scale, from the exponent field of its largest magnitude."""
    bits = amax.view(torch.int32)
    e = bits >> 23
    if rule == CEIL:
        e = e + ((bits & 0x7FFFFF) > 0x400000)
    return (e - 2).clamp_(min=0)


def _power(code):
    """2^(code - 127) in float32; code 0 is the subnormal 2^-127."""
    return torch.where(code > 0, code << 23, 0x400000).view(torch.float32)


def _blocks(v, to=BLOCK):
    """float32, the last axis padded with zeros to a multiple of `to`, split into blocks."""
    v = v.float()
    v = torch.nn.functional.pad(v, (0, -v.shape[-1] % to))
    return v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)


def _round(v, rule):
    """Blocks -> (E2M1 magnitudes with sign, scale codes)."""
    code = _scale(v.abs().amax(-1, keepdim=True), rule)
    u = v / _power(code)
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp_(max=6)
    return torch.copysign(q, u), code


def _quantized(v, rule):
    """Values of the 1 x 32 quantisation along the last axis, in float32."""
    q, code = _round(_blocks(v), rule)
    return (q * _power(code)).flatten(-2)[..., :v.shape[-1]]


def _pack(w):
    """Packed copy of w along its last axis: codes (element 2i in the low nibble) and scales."""
    q, code = _round(_blocks(w, PAD), FLOOR)
    a = q.abs()
    c = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = (c | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), code.squeeze(-1).to(torch.uint8)


def _decoded(codes, scales, k):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                        device=codes.device)
    pairs = torch.stack([grid.repeat(16), grid.repeat_interleave(16)], dim=-1)
    v = pairs[codes.int()].flatten(-2)
    v = v.reshape(*scales.shape, BLOCK) * _power(scales.int()).unsqueeze(-1)
    return v.flatten(-2)[..., :k]


def _by_group(x, offsets, most):
    """Rows -> [groups][most rows], zero where a group has fewer; also each row's place there."""
    rows = torch.arange(x.shape[0], device=x.device)
    group = torch.searchsorted(offsets[1:].contiguous(), rows.int(), right=True)
    place = group * most + rows - offsets[group]
    padded = x.new_zeros((offsets.numel() - 1) * most, x.shape[1])
    padded[place] = x
    return padded.view(-1, most, x.shape[1]), place


def _plain(s):
    case, x = s["case"], s["x"]
    kind, rule, dtype = case["kind"], case["rule"], s["x"].dtype
    offsets = s.get("offsets")
    if kind == "quantize":
        got = [_quantized(x, rule).to(dtype)]
        if case["col"]:
            if offsets is None:
                got.append(_quantized(x.t(), rule).to(dtype))
            else:
                most = -(-s["most"] // BLOCK) * BLOCK
                padded, place = _by_group(x.float(), offsets, most)
                q = _quantized(padded.transpose(1, 2), rule).transpose(1, 2)
                got.append(q.reshape(-1, x.shape[1])[place].t().to(dtype).contiguous())
        return got
    if kind == "linear":
        w = _decoded(s["w_codes"], s["w_scales"], case["cols"])
        return (_quantized(x, rule) @ w.t()).to(dtype)
    if kind == "experts":
        w = _decoded(s["w_codes"], s["w_scales"], case["cols"])
        padded, place = _by_group(_quantized(x, rule), offsets, s["most"])
        y = torch.bmm(padded, w.transpose(1, 2).contiguous())
        return y.view(-1, case["out"])[place].to(dtype)
    w, dy = s["w"], s["dy"]
    xr, wr, dyr = _quantized(x, rule), _quantized(w, rule), _quantized(dy, rule)
    wc = _quantized(w.transpose(-1, -2), rule)
    if kind == "train":
        dw = _quantized(dy.t(), rule) @ _quantized(x.t(), rule).t()
        return [(xr @ wr.t()).to(dtype), (dyr @ wc.t()).to(dtype), dw]
    most = -(-s["most"] // BLOCK) * BLOCK
    xp, place = _by_group(xr, offsets, most)
    dyp, _ = _by_group(dyr, offsets, most)
    y = torch.bmm(xp, wr.transpose(1, 2).contiguous()).view(-1, case["out"])[place]
    dx = torch.bmm(dyp, wc.transpose(1, 2).contiguous()).view(-1, case["cols"])[place]
    xc = _quantized(_by_group(x.float(), offsets, most)[0].transpose(1, 2), rule)
    dyc = _quantized(_by_group(dy.float(), offsets, most)[0].transpose(1, 2), rule)
    dw = torch.bmm(dyc, xc.transpose(1, 2).contiguous())
    return [y.to(dtype), dx.to(dtype), dw]


# ---------------------------------------------------------------------------- the library
def _library(s):
    import nvfp4_block_scaled_quantize_amd as nv
    case, x = s["case"], s["x"]
    kind, rule, dtype = case["kind"], case["rule"], s["x"].dtype
    offsets = s.get("offsets")
    if kind == "quantize":
        p = nv.mxfp4_quant_params(rowwise=True, colwise=case["col"], scale_rule=rule)
        row, col = nv.mxfp4_quantize(x, p, offsets=offsets)
        got = [nv.mxfp4_dequantize(row, dtype)]
        if case["col"]:
            got.append(nv.mxfp4_dequantize(col, dtype, offsets=offsets))
        return got
    if kind in ("linear", "experts"):
        w = nv.MXTensor(s["w_codes"], s["w_scales"], case["cols"])
        return nv.mxfp4_linear(x, w, offsets=offsets, scale_rule=rule, out_dtype=dtype)
    p = nv.mxfp4_quant_params(rowwise=True, colwise=True, scale_rule=rule)
    xr, xc = nv.mxfp4_quantize(x, p, offsets=offsets)
    wr, wc = nv.mxfp4_quantize(s["w"], p)
    dyr, dyc = nv.mxfp4_quantize(s["dy"], p, offsets=offsets)
    if kind == "train":
        return [nv.mxfp4_gemm(xr, wr, out_dtype=dtype), nv.mxfp4_gemm(dyr, wc, out_dtype=dtype),
                nv.mxfp4_gemm(dyc, xc)]
    return [nv.mxfp4_gemm_grouped(xr, wr, offsets, out_dtype=dtype),
            nv.mxfp4_gemm_grouped(dyr, wc, offsets, out_dtype=dtype),
            nv.mxfp4_gemm_grouped_wgrad(dyc, xc, offsets)]


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------- work
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    t, k = case["rows"], case["cols"]
    if case["kind"] == "quantize":
        # X once, the decoded values of each copy once
        return {"bytes": t * k * size * (3 if case["col"] else 2), "flops": 0}
    n, groups = case["out"], case.get("groups", 0)
    busy = sum(c > 0 for c in _counts(t, groups, case["busy"])) if groups else 1
    if case["kind"] in ("linear", "experts"):
        packed = n * (k + -k % PAD) * 17 // 32
        return {"bytes": (t * k + t * n) * size + busy * packed, "flops": 2 * t * n * k}
    # X, dY and the weights of experts with rows once; Y and dX; float32 dW of every expert
    return {"bytes": 2 * (t * k + t * n) * size + busy * n * k * size + max(groups, 1) * n * k * 4,
            "flops": 6 * t * n * k}


# ---------------------------------------------------------------------------- 64 bits
def _exact_values(v, rule):
    """1 x 32 quantisation along the last axis in float64: scale from the binary logarithm's
    integer part (frexp), nearest grid point by counting the midpoints passed, ties to even."""
    k = v.shape[-1]
    v = v.double()
    out = torch.empty_like(v)
    whole = k // BLOCK * BLOCK
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    for part in (slice(0, whole), slice(whole, k)):
        b = v[..., part]
        if b.shape[-1] == 0:
            continue
        b = b.reshape(*b.shape[:-1], -1, min(BLOCK, b.shape[-1]))
        m, e = torch.frexp(b.abs().amax(-1, keepdim=True))     # amax = m 2^e, m in [1/2, 1)
        # floor: floor(log2 amax) = e - 1; ceil: 6 2^p >= amax, 6 = 0.75 2^3
        p = e - 3 if rule == FLOOR else torch.where(m <= 0.75, e - 3, e - 2)
        p = torch.where(m == 0, torch.full_like(p, -127), p.clamp(min=-127))
        scale = ((p.long() + 1023) << 52).view(torch.float64)   # 2^p, exactly
        a = b.abs() / scale
        index = torch.zeros_like(a, dtype=torch.int64)
        for i in range(7):
            mid = (grid[i] + grid[i + 1]) / 2
            index += (a > mid) if i % 2 == 0 else (a >= mid)
        out[..., part] = torch.copysign(grid[index] * scale, b).flatten(-2)
    return out


def exact(case, seed):
    if 2 * case["rows"] * case["cols"] * case.get("out", 1) > 2e12:
        return None
    s = _inputs(case, seed)
    x, rule, kind = s["x"], case["rule"], case["kind"]
    groups = case.get("groups", 0)
    ends = s["offsets"].tolist() if groups else [0, case["rows"]]
    spans = list(zip(ends[:-1], ends[1:]))

    def columns(v):   # blocks along the rows, starting anew at each span
        return torch.cat([_exact_values(v[a:b].t(), rule) for a, b in spans], dim=1)

    xr = _exact_values(x, rule)
    if kind == "quantize":
        return [xr, columns(x)] if case["col"] else [xr]
    w = s["w"] if groups else s["w"][None]
    wr = _exact_values(w, rule if "train" in kind else FLOOR)
    y = torch.cat([xr[a:b] @ wr[g].t() for g, (a, b) in enumerate(spans)])
    if "train" not in kind:
        return y
    wc = _exact_values(w.transpose(1, 2), rule)
    dyr, dyc, xc = _exact_values(s["dy"], rule), columns(s["dy"]), columns(x)
    dx = torch.cat([dyr[a:b] @ wc[g].t() for g, (a, b) in enumerate(spans)])
    dw = torch.stack([dyc[:, a:b] @ xc[:, a:b].t() for a, b in spans])
    return [y, dx, dw if groups else dw[0]]
