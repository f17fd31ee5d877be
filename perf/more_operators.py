"""What is measured of the gated feed-forward block on MXFP4 products and of the 8-bit (MXFP8)
activation checkpoints that its backward pass reads.

``run`` computes each operator in plain torch (``own`` false: float32 throughout, rounded once
at the end) or through the library (``own`` true).  ``exact`` computes it in 64 bits.

The block: G = X Wg^T, U = X Wu^T, H = act(G) * U, Y = H W2^T, with X, W = [Wg; Wu], H and W2
as MXFP4 operands (E2M1 elements, an E8M0 scale per 32).  A checkpoint is MXFP8: E4M3 elements,
an E8M0 scale per 32, the smallest power of two by which nothing saturates.
"""
import math

import torch

own = False

BLOCK = 32       # elements per scale
PAD = 128        # the copies' K extent is padded to a multiple of this with zero codes
FLOOR, CEIL = 0, 1
ROOT = math.sqrt(2 / math.pi)


# ---------------------------------------------------------------------------- cases
def listed():
    """kind: checkpoint (values of an 8-bit checkpoint), reuse (MXFP4 copies made of one), gated
    (serving: H from activations), ffn (the block's forward; train: with the checkpoint of G and
    U), backward (dG, dU and H from dY, or from dH where out is 0)."""
    return [
        # a layer's input kept for the backward pass
        {"name": "checkpoint_hidden", "kind": "checkpoint", "rows": 8192, "cols": 4096,
         "dtype": "bf16", "pad": 0},
        # float32 view into a wider buffer, no extent a multiple of anything
        {"name": "checkpoint_odd", "kind": "checkpoint", "rows": 1021, "cols": 1531,
         "dtype": "f32", "pad": 5},
        # the kept input becomes the operands of the backward pass's products
        {"name": "reuse_hidden", "kind": "reuse", "rows": 8192, "cols": 4096, "dtype": "bf16",
         "rule": CEIL, "groups": 0, "busy": 0},
        # the same of tokens sorted by expert: columnwise blocks end where an expert's rows end
        {"name": "reuse_experts", "kind": "reuse", "rows": 12001, "cols": 2048, "dtype": "bf16",
         "rule": CEIL, "groups": 64, "busy": 57},
        # one token through a gated layer
        {"name": "gated_token", "kind": "gated", "rows": 1, "cols": 4096, "mid": 9216,
         "dtype": "bf16", "act": "silu", "groups": 0, "busy": 0},
        # a batch of decoding sequences, odd sizes
        {"name": "gated_batch", "kind": "gated", "rows": 77, "cols": 2056, "mid": 4999,
         "dtype": "bf16", "act": "gelu", "groups": 0, "busy": 0},
        # a few decoding tokens, each routed to some of the experts
        {"name": "gated_experts", "kind": "gated", "rows": 24, "cols": 2048, "mid": 1536,
         "dtype": "bf16", "act": "silu", "groups": 32, "busy": 17},
        # a prompt of 8192 tokens through the whole block
        {"name": "ffn_prompt", "kind": "ffn", "rows": 8192, "cols": 4096, "mid": 9216, "out": 4096,
         "dtype": "bf16", "act": "silu", "rule": FLOOR, "train": False, "groups": 0, "busy": 0},
        # the forward of a training step of an expert block
        {"name": "ffn_experts_train", "kind": "ffn", "rows": 8191, "cols": 2048, "mid": 1536, "out": 2048,
         "dtype": "bf16", "act": "silu", "rule": CEIL, "train": True, "groups": 16, "busy": 15},
        # the backward pass through the down projection and the gate
        {"name": "backward_layer", "kind": "backward", "rows": 8192, "mid": 9216, "out": 4096,
         "dtype": "bf16", "act": "silu", "rule": CEIL, "groups": 0, "busy": 0},
        # the same of an expert block
        {"name": "backward_experts", "kind": "backward", "rows": 8191, "mid": 1536, "out": 2048,
         "dtype": "bf16", "act": "silu", "rule": CEIL, "groups": 16, "busy": 15},
        # a small float32 layer of odd sizes whose dH another product made
        {"name": "backward_odd", "kind": "backward", "rows": 1000, "mid": 777, "out": 0,
         "dtype": "f32", "act": "gelu", "rule": CEIL, "groups": 0, "busy": 0},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def extent(lo, hi):   # ordinary extents are multiples of 64, some are odd
        n = size(lo, hi)
        return n if rng.random() < 0.35 else max(64, n // 64 * 64)

    kind = rng.choice(["checkpoint", "reuse", "gated", "ffn", "backward", "backward"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if kind == "checkpoint":
        return {"kind": kind, "rows": size(1, 8192), "cols": extent(64, 9216), "dtype": dtype,
                "pad": rng.choice([0, 0, 3, 64])}
    groups = rng.choice([0, 0, size(2, 32)])
    c = {"kind": kind, "rows": size(1, 8192), "dtype": dtype, "groups": groups,
         "busy": max(1, groups - rng.randrange(0, 4)) if groups else 0}
    if kind == "reuse":
        return c | {"cols": extent(64, 8192), "rule": rng.choice([FLOOR, CEIL])}
    most = 2048 if groups else 6144
    c |= {"mid": extent(64, most), "act": rng.choice(["silu", "silu", "gelu"])}
    if kind != "backward":
        c["cols"] = extent(256, 2048 if groups else 4096)
    if kind == "gated":
        return c
    c |= {"out": extent(256, 2048 if groups else 4096), "rule": rng.choice([FLOOR, CEIL])}
    if kind == "ffn":
        return c | {"train": rng.random() < 0.6}
    if not groups and rng.random() < 0.4:
        c["out"] = 0
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
    """The operands before they are packed."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, kind, rows = _DTYPE[case["dtype"]], case["kind"], case["rows"]
    groups, s = case.get("groups", 0), {}
    if groups:
        order = torch.randperm(groups, generator=torch.Generator().manual_seed(int(seed))).tolist()
        counts = _counts(rows, groups, case["busy"])
        counts = [counts[i] for i in order]
        s["most"] = max(counts)
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")

    def weights(n, k):
        return 0.02 * torch.randn((groups, n, k) if groups else (n, k), generator=gen, device="cuda")

    if kind != "backward":
        s["x"] = _activations(rows, case["cols"], dtype, gen, case.get("pad", 0))
    if kind in ("gated", "ffn"):
        s["w"] = weights(2 * case["mid"], case["cols"])
    if kind == "backward":
        # G and U of a layer: of the size that such weights make of such activations
        s["gu"] = 2 * torch.randn(2, rows, case["mid"], generator=gen, device="cuda")
        name, width = ("dy", case["out"]) if case["out"] else ("dh", case["mid"])
        s[name] = _gradients(rows, width, dtype, gen)
    if case.get("out"):
        s["w2"] = weights(case["out"], case["mid"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    kind = case["kind"]
    if kind in ("gated", "ffn"):        # weights are held packed, as a server or a step keeps them
        s["w"] = _pack(s["w"])
    if kind == "ffn":
        s["w2"] = _pack(s["w2"])
    if kind == "backward":
        s["gu"] = _pack8(s["gu"])
        if case["out"]:                 # the columnwise copy: W2^T in blocks along its rows, rows side by side
            s["w2"] = tuple(t.contiguous() for t in _pack(s["w2"].transpose(-1, -2)))
    if kind == "reuse":
        s["x8"] = _pack8(s.pop("x"))
    return s


# ---------------------------------------------------------------------------- plain form
def _power(code):
    """2^(code - 127) in float32; code 0 is the subnormal 2^-127."""
    return torch.where(code > 0, code << 23, 0x400000).view(torch.float32)


def _code(blocks, exponent, above):
    """E8M0 codes: the exponent field of each block's largest magnitude less `exponent`, one more
    where the fraction field exceeds `above`."""
    bits = blocks.abs().amax(-1, keepdim=True).view(torch.int32)
    return ((bits >> 23) + ((bits & 0x7FFFFF) > above) - exponent).clamp_(min=0)


def _blocks(v, to=BLOCK):
    """float32, the last axis padded with zeros to a multiple of `to`, split into blocks."""
    v = v.float()
    v = torch.nn.functional.pad(v, (0, -v.shape[-1] % to))
    return v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)


def _round4(v, rule):
    """Blocks -> (E2M1 values with sign, scale codes)."""
    code = _code(v, 2, 0x400000 if rule == CEIL else 0x7FFFFF)
    u = v / _power(code)
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp_(max=6), u), code


def _round8(v):
    """Blocks -> (E4M3 values with sign, scale codes)."""
    code = _code(v, 8, 0x600000)
    u = v / _power(code)
    step = _power(((u.abs().view(torch.int32) >> 23) - 3).clamp_(min=127 - 9))   # 2^-9 below 2^-6
    return torch.copysign(torch.round(u.abs() / step) * step, u), code


def _quantized(v, rule):
    """Values of the MXFP4 quantisation along the last axis, in float32."""
    q, code = _round4(_blocks(v), rule)
    return (q * _power(code)).flatten(-2)[..., :v.shape[-1]]


def _quantized8(v):
    """Values of the MXFP8 quantisation along the last axis, in float32."""
    q, code = _round8(_blocks(v))
    return (q * _power(code)).flatten(-2)[..., :v.shape[-1]]


def _pack(w):
    """MXFP4 copy of w along its last axis: codes (element 2i in the low nibble) and scales."""
    q, code = _round4(_blocks(w, PAD), FLOOR)
    a = q.abs()
    c = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = (c | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), code.squeeze(-1).to(torch.uint8)


def _pack8(v):
    """MXFP8 copy along the last axis: a byte an element, and scales."""
    q, code = _round8(_blocks(v, PAD))
    return q.flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8), code.squeeze(-1).to(torch.uint8)


def _decoded(packed, k):
    codes, scales = packed
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                        device=codes.device)
    pairs = torch.stack([grid.repeat(16), grid.repeat_interleave(16)], dim=-1)
    v = pairs[codes.int()].flatten(-2)
    v = v.reshape(*scales.shape, BLOCK) * _power(scales.int()).unsqueeze(-1)
    return v.flatten(-2)[..., :k]


def _decoded8(packed, k):
    codes, scales = packed
    v = codes.view(torch.float8_e4m3fn).float().reshape(*scales.shape, BLOCK)
    return (v * _power(scales.int()).unsqueeze(-1)).flatten(-2)[..., :k]


def _by_group(x, offsets, most):
    """Rows -> [groups][most rows], zero where a group has fewer; also each row's place there."""
    rows = torch.arange(x.shape[0], device=x.device)
    group = torch.searchsorted(offsets[1:].contiguous(), rows.int(), right=True)
    place = group * most + rows - offsets[group]
    padded = x.new_zeros((offsets.numel() - 1) * most, x.shape[1])
    padded[place] = x
    return padded.view(-1, most, x.shape[1]), place


def _product(x, w, s):
    """x w^T, each group's rows with its own w where there are groups."""
    if "offsets" not in s:
        return x @ w.t()
    padded, place = _by_group(x, s["offsets"], s["most"])
    return torch.bmm(padded, w.transpose(1, 2).contiguous()).view(-1, w.shape[1])[place]


def _act(g, name):
    """The activation and its derivative."""
    if name == "silu":
        t = torch.sigmoid(g)
        return g * t, t * (1 + g * (1 - t))
    t = torch.tanh(ROOT * (g + 0.044715 * g ** 3))
    slope = ROOT * (1 + 3 * 0.044715 * g * g)
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * slope


def _plain(s):
    case, kind, dtype = s["case"], s["case"]["kind"], _DTYPE[s["case"]["dtype"]]
    if kind == "checkpoint":
        return _quantized8(s["x"]).to(dtype)
    if kind == "reuse":
        x, rule = _decoded8(s["x8"], case["cols"]), case["rule"]
        row = _quantized(x, rule).to(dtype)
        if "offsets" not in s:
            return [row, _quantized(x.t(), rule).to(dtype)]
        most = -(-s["most"] // BLOCK) * BLOCK
        padded, place = _by_group(x, s["offsets"], most)
        q = _quantized(padded.transpose(1, 2), rule).transpose(1, 2)
        return [row, q.reshape(-1, x.shape[1])[place].t().to(dtype).contiguous()]
    if kind == "backward":
        g, u = _decoded8(s["gu"], case["mid"])
        if case["out"]:
            w2 = _decoded(s["w2"], case["out"])
            dh = _product(_quantized(s["dy"], case["rule"]), w2, s)
        else:
            dh = s["dh"].float()
        a, slope = _act(g, case["act"])
        return [torch.cat([dh * u * slope, dh * a], dim=1).to(dtype), (a * u).to(dtype)]
    x = _quantized(s["x"], case.get("rule", FLOOR))
    gu = _product(x, _decoded(s["w"], case["cols"]), s)
    g, u = gu[:, :case["mid"]], gu[:, case["mid"]:]
    h = _act(g, case["act"])[0] * u
    if kind == "gated":
        return h.to(dtype)
    y = _product(_quantized(h, case["rule"]), _decoded(s["w2"], case["mid"]), s).to(torch.bfloat16)
    if not case["train"]:
        return y
    # the values of a checkpoint of bfloat16's range fit into bfloat16
    return [y, _quantized8(g).to(torch.bfloat16), _quantized8(u).to(torch.bfloat16)]


# ---------------------------------------------------------------------------- the library
def _library(s):
    import nvfp4_block_scaled_quantize_amd as nv
    case, kind, dtype = s["case"], s["case"]["kind"], _DTYPE[s["case"]["dtype"]]
    offsets = s.get("offsets")
    if kind == "checkpoint":
        return nv.mxfp8_dequantize(nv.mxfp8_quantize(s["x"]), dtype)
    if kind == "reuse":
        p = nv.mxfp4_quant_params(rowwise=True, colwise=True, scale_rule=case["rule"])
        row, col = nv.mxfp8_to_mxfp4(nv.MX8Tensor(*s["x8"], case["cols"]), p, offsets=offsets)
        return [nv.mxfp4_dequantize(row, dtype), nv.mxfp4_dequantize(col, dtype, offsets=offsets)]
    act = nv.MXFP4_GELU if case["act"] == "gelu" else nv.MXFP4_SILU
    if kind == "gated":
        return nv.mxfp4_gated_linear(s["x"], nv.MXTensor(*s["w"], case["cols"]), offsets=offsets,
                                     activation=act)
    p = nv.mxfp4_quant_params(scale_rule=case["rule"])
    if kind == "ffn":
        x, _ = nv.mxfp4_quantize(s["x"], p)
        _, h, kept = nv.mxfp4_gated(x, nv.MXTensor(*s["w"], case["cols"]), offsets=offsets, activation=act,
                                    out_dtype=None, packed=True, scale_rule=case["rule"],
                                    checkpoint=case["train"])
        w2 = nv.MXTensor(*s["w2"], case["mid"])
        y = (nv.mxfp4_gemm(h, w2, out_dtype=torch.bfloat16) if offsets is None else
             nv.mxfp4_gemm_grouped(h, w2, offsets, out_dtype=torch.bfloat16))
        if not case["train"]:
            return y
        values = nv.mxfp8_dequantize(kept, torch.bfloat16)
        return [y, values[0], values[1]]
    kept = nv.MX8Tensor(*s["gu"], case["mid"])
    if not case["out"]:
        return list(nv.mxfp8_gated_backward(s["dh"], kept, activation=act, h=True))
    dy, _ = nv.mxfp4_quantize(s["dy"], p)
    return list(nv.mxfp4_gated_backward(dy, nv.MXTensor(*s["w2"], case["out"]), kept, offsets=offsets,
                                        activation=act, out_dtype=dtype, h=True))


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------- work
def work(case):
    size, kind, t = (2 if case["dtype"] == "bf16" else 4), case["kind"], case["rows"]
    if kind == "checkpoint":    # X once, its checkpoint's values once
        return {"bytes": 2 * t * case["cols"] * size, "flops": 0}
    if kind == "reuse":         # the checkpoint, the values of two copies
        return {"bytes": t * case["cols"] * (33 / 32 + 2 * size), "flops": 0}
    groups, n = case["groups"], case["mid"]
    busy = sum(c > 0 for c in _counts(t, groups, case["busy"])) if groups else 1

    def packed(rows, k):
        return rows * (k + -k % PAD) * 17 // 32

    kept = 2 * t * n * 33 // 32
    if kind == "backward":
        d = case["out"]
        given = t * d * size + busy * packed(n, d) if d else t * n * size
        return {"bytes": given + kept + 3 * t * n * size, "flops": 2 * t * n * d}
    k = case["cols"]
    need, flops = t * k * size + busy * packed(2 * n, k), 4 * t * n * k
    if kind == "gated":
        return {"bytes": need + t * n * size, "flops": flops}
    d = case["out"]
    values = 2 * t * n * 2 if case["train"] else 0
    return {"bytes": need + busy * packed(d, n) + t * d * 2 + values, "flops": flops + 2 * t * n * d}


# ---------------------------------------------------------------------------- 64 bits
def _exact_blocks(v, of):
    """`of` applied to the blocks of v along its last axis, a shorter one at its end."""
    k, v = v.shape[-1], v.double()
    out = torch.empty_like(v)
    whole = k // BLOCK * BLOCK
    for part in (slice(0, whole), slice(whole, k)):
        b = v[..., part]
        if b.shape[-1]:
            out[..., part] = of(b.reshape(*b.shape[:-1], -1, min(BLOCK, b.shape[-1]))).flatten(-2)
    return out


def _two_to(p):
    return ((p.long() + 1023) << 52).view(torch.float64)


def _exact4(v, rule):
    """MXFP4: scale from the binary logarithm's integer part (frexp), nearest grid point by
    counting the midpoints passed, ties to even."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)

    def of(b):
        m, e = torch.frexp(b.abs().amax(-1, keepdim=True))     # amax = m 2^e, m in [1/2, 1)
        # floor: floor(log2 amax) = e - 1; ceil: 6 2^p >= amax, 6 = 0.75 2^3
        p = e - 3 if rule == FLOOR else torch.where(m <= 0.75, e - 3, e - 2)
        scale = _two_to(torch.where(m == 0, torch.full_like(p, -127), p.clamp(min=-127)))
        a = b.abs() / scale
        index = torch.zeros_like(a, dtype=torch.int64)
        for i in range(7):
            mid = (grid[i] + grid[i + 1]) / 2
            index += (a > mid) if i % 2 == 0 else (a >= mid)
        return torch.copysign(grid[index] * scale, b)

    return _exact_blocks(v, of)


def _exact8(v):
    """MXFP8: 448 2^p >= amax with 448 = 0.875 2^9; a value m 2^e (m in [1/2, 1)) of the grid has
    four significant bits, or steps of 2^-9 below 2^-6."""
    def of(b):
        m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
        p = torch.where(m <= 0.875, e - 9, e - 8)
        scale = _two_to(torch.where(m == 0, torch.full_like(p, -127), p.clamp(min=-127)))
        step = _two_to(torch.frexp(b / scale)[1].clamp(min=-5) - 4)
        n, f = torch.div(b / scale, step).trunc(), (b / scale / step).frac().abs()
        up = (f > 0.5) | ((f == 0.5) & (n % 2 != 0))
        return (n + torch.copysign(up.double(), b)) * step * scale

    return _exact_blocks(v, of)


def _exact_act(g, name):
    if name == "silu":
        t = 1 / (1 + torch.exp(-g))
        return g * t, t + g * t * (1 - t)
    # 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))
    t = 1 / (1 + torch.exp(-2 * ROOT * (g + 0.044715 * g * g * g)))
    return g * t, t + g * t * (1 - t) * 2 * ROOT * (1 + 0.134145 * g * g)


def exact(case, seed):
    s, kind = _inputs(case, seed), case["kind"]
    ends = s["offsets"].tolist() if "offsets" in s else [0, case["rows"]]
    spans = list(zip(ends[:-1], ends[1:]))

    def product(x, w):      # each span's rows with its w
        w = w if "offsets" in s else w[None]
        return torch.cat([x[a:b] @ w[i].t() for i, (a, b) in enumerate(spans)])

    if kind == "checkpoint":
        return _exact8(s["x"])
    if kind == "reuse":
        x, rule = _exact8(s["x"]), case["rule"]
        return [_exact4(x, rule), torch.cat([_exact4(x[a:b].t(), rule) for a, b in spans], dim=1)]
    if kind == "backward":
        g, u = _exact8(s["gu"])
        if case["out"]:
            dh = product(_exact4(s["dy"], case["rule"]), _exact4(s["w2"].transpose(-1, -2), FLOOR))
        else:
            dh = s["dh"].double()
        a, slope = _exact_act(g, case["act"])
        return [torch.cat([dh * u * slope, dh * a], dim=1), a * u]
    w = _exact4(s["w"], FLOOR)
    x = _exact4(s["x"], case.get("rule", FLOOR))
    n = case["mid"]
    g, u = product(x, w[..., :n, :]), product(x, w[..., n:, :])
    h = _exact_act(g, case["act"])[0] * u
    if kind == "gated":
        return h
    y = product(_exact4(h, case["rule"]), _exact4(s["w2"], FLOOR))
    return [y, _exact8(g), _exact8(u)] if case["train"] else y
