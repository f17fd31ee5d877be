"""8-bit activation checkpoints on the GPU against the plain 64-bit implementation, bit for bit: made,
decoded, turned into MXFP4 copies; and the gated product's gradients from them."""
import numpy as np
import pytest
import torch

import mxffn_reference as ref
import mxfp4_reference as ref4
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load_library()
    return nv


DTYPES = [torch.bfloat16, torch.float32]
SIZES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 127), (4, 128), (7, 129), (1, 5000), (130, 65), (257, 640), (64, 1531),
         (1000, 96), (4099, 33)]


def values_of(shape, seed, dtype):
    """Magnitudes over many binades, some zeros."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=dev()) * torch.exp(3 * torch.randn(shape, generator=g, device=dev()))
    x[torch.rand(shape, generator=g, device=dev()) < 0.05] = 0
    return x.to(dtype)


def same(q, want, what):
    codes, scales = (torch.from_numpy(w).to(dev()) for w in want)
    assert torch.equal(q.scales, scales), f"{what}: {int((q.scales != scales).sum())} scales differ"
    assert torch.equal(q.codes, codes), f"{what}: {int((q.codes != codes).sum())} codes differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_and_decode(nv, rows, cols, dtype):
    print(f"mx8 {rows}x{cols} {dtype}", flush=True)
    wide = values_of((rows, cols + 5), rows * 7 + cols, dtype)
    for x in (wide[:, :cols], wide[:, 3:3 + cols], wide[:, :cols].contiguous()):
        want = ref.quantize_rows(x.double().cpu().numpy())
        out = nv.MX8Tensor.empty(rows, cols, dev())
        out.codes.fill_(0x55), out.scales.fill_(0x55)           # padding is written too
        assert nv.mxfp8_quantize(x, out) is out
        same(out, want, "quantize")
    v = torch.from_numpy(ref.decode(*want)[:, :cols]).to(dev())
    for dt in DTYPES:
        got = nv.mxfp8_dequantize(out, dt)
        assert got.dtype == dt and torch.equal(got.double(), v)         # E4M3 fits into bfloat16
        for at, pitch in ((0, cols), (1, cols + 1), (2, cols + 6), (3, cols + 3)):
            buf = torch.full((rows + 2, pitch + 4), 7.0, dtype=dt, device=dev())
            nv.mxfp8_dequantize(out, out=buf[1:-1, at:at + cols])
            assert torch.equal(buf[1:-1, at:at + cols], got)
            buf[1:-1, at:at + cols] = 7.0
            assert (buf == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_code_and_scale(nv, dtype):
    """All 254 finite codes at scales over the whole range decode to their values, in float32 exactly, in
    bfloat16 rounded once; 255 to NaN, and the two NaN codes."""
    codes = torch.arange(256, dtype=torch.uint8, device=dev()).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8, device=dev())[:, None].repeat(1, 8)
    q = nv.MX8Tensor(codes, scales, 256)
    want = torch.from_numpy(ref.decode(codes.cpu().numpy(), scales.cpu().numpy())).to(dev())
    got = nv.mxfp8_dequantize(q, dtype)
    want = want.float().to(dtype)      # float32 holds them all up to 2^128
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0, 1, -1), want.nan_to_num(0, 1, -1))


@pytest.mark.parametrize("dtype", DTYPES)
def test_borders_and_special_values(nv, dtype):
    """Every border of the scale and the ties of every code; zeros of both signs, subnormals, the
    largest value; blocks with an infinity or a NaN."""
    grid = torch.tensor(ref.GRID, dtype=torch.float64)
    ties = (grid[1:] + grid[:-1]) / 2
    row = torch.cat([grid, -grid, ties, -ties])
    row = row[:-(-row.numel() // 31) * 31 or None]
    row = torch.nn.functional.pad(row, (0, -row.numel() % 31)).reshape(-1, 31)
    row = torch.cat([torch.full((row.shape[0], 1), 448.0, dtype=torch.float64), row], 1).reshape(1, -1)
    x = torch.cat([row * 2.0 ** p for p in (-126, -60, -8, -1, 0, 1, 50, 118)])
    more = torch.zeros(12, row.shape[1], dtype=torch.float64)
    big = torch.finfo(dtype).max
    for i, v in enumerate([0.0, -0.0, torch.finfo(dtype).tiny, 2.0 ** -133, big, -big, float("inf"), -float("inf"), float("nan"),
                           1.75, 1.7578125, 2.0 ** -118]):
        more[i, i] = v
        more[i, 33:40] = 3.0
    x = torch.cat([x, more]).to(dtype).to(dev())
    same(nv.mxfp8_quantize(x), ref.quantize_rows(x.double().cpu().numpy()), "borders")


@pytest.mark.parametrize("dtype", DTYPES)
def test_stacks(nv, dtype):
    x = values_of((3, 9, 70), 3, dtype)
    for v in (x, x[::2], x.transpose(0, 1), values_of((40, 2, 70), 4, dtype).transpose(0, 1)[:, 3:]):
        q = nv.mxfp8_quantize(v)
        assert q.shape == tuple(v.shape)
        want = ref.quantize_rows(v.double().cpu().numpy().reshape(-1, 70))
        n = v.shape[0] * v.shape[1]
        same(nv.MX8Tensor(q.codes.view(n, 128), q.scales.view(n, 4), 70), want, "stack")
        assert torch.equal(nv.mxfp8_dequantize(q).double().cpu().view(n, 70), torch.from_numpy(ref.decode(*want)[:, :70]))


def test_empty(nv):
    for shape in ((0, 5), (5, 0), (0, 4, 5), (2, 0, 5)):
        q = nv.mxfp8_quantize(torch.empty(shape, device=dev()))
        assert q.shape == shape and nv.mxfp8_dequantize(q).shape == shape
    q = nv.MX8Tensor.empty((2, 0), 5, dev())
    dgu, h = nv.mxfp8_gated_backward(torch.empty(0, 5, device=dev()), q, h=True)
    assert dgu.shape == (0, 10) and h.shape == (0, 5)


def equal_copies(a, b, used=None):
    if a is None or b is None:
        return a is b
    return torch.equal(a.codes[..., :used and used // 2], b.codes[..., :used and used // 2]) and \
        torch.equal(a.scales[..., :used and used // 32], b.scales[..., :used and used // 32])


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 40), (33, 128), (130, 129), (257, 700), (600, 2048)])
@pytest.mark.parametrize("rule", [ref4.FLOOR, ref4.CEIL])
def test_to_mxfp4_is_quantize_of_the_values(nv, rows, cols, rule):
    print(f"to mxfp4 {rows}x{cols} {rule}", flush=True)
    for lead in ((rows,), (3, rows)):
        q = nv.mxfp8_quantize(values_of((*lead, cols), rows, torch.float32))
        q.codes[..., cols:] = 0x7E      # what lies behind a row's end is not read
        v = nv.mxfp8_dequantize(q, torch.bfloat16)
        for row, col in ((True, False), (False, True), (True, True)):
            for sr in (nv.NVFP4_RNE, nv.NVFP4_SR):
                p = nv.mxfp4_quant_params(row, col, rule, sr, sr, 77)
                got, want = nv.mxfp8_to_mxfp4(q, p), nv.mxfp4_quantize(v, p)
                assert all(equal_copies(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,cols,offsets", [(5, 40, [0, 2, 2, 5]), (700, 130, [0, 1, 129, 400, 690]), (900, 96, [3, 1000, 5])])
def test_to_mxfp4_grouped(nv, rows, cols, offsets):
    q = nv.mxfp8_quantize(values_of((rows, cols), rows, torch.bfloat16))
    off = torch.tensor(offsets, dtype=torch.int32, device=dev())
    used = ref4.grouped_positions(offsets, rows)[2]
    for sr in (nv.NVFP4_RNE, nv.NVFP4_SR):
        p = nv.mxfp4_quant_params(True, True, ref4.CEIL, sr, sr, 5)
        got = nv.mxfp8_to_mxfp4(q, p, offsets=off)
        want = nv.mxfp4_quantize(nv.mxfp8_dequantize(q, torch.bfloat16), p, offsets=off)
        assert equal_copies(got[0], want[0]) and equal_copies(got[1], want[1], used)


def test_to_mxfp4_past_the_caches(nv):
    """A checkpoint of more than 128 MB, which is read as a stream."""
    q = nv.MX8Tensor(torch.randint(0, 127, (16500, 8192), dtype=torch.uint8, device=dev()),
                     torch.randint(100, 140, (16500, 256), dtype=torch.uint8, device=dev()), 8150)
    p = nv.mxfp4_quant_params(True, True)
    got, want = nv.mxfp8_to_mxfp4(q, p), nv.mxfp4_quantize(nv.mxfp8_dequantize(q, torch.bfloat16), p)
    assert all(equal_copies(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("nan", [False, True])
def test_to_mxfp4_of_every_code_and_scale(nv, nan):
    """Scale r in row r, and so 32 neighbouring ones in a columnwise block; shuffled rows in a second matrix."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    if not nan:
        codes[(codes & 0x7F) == 0x7F] = 0
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    order = torch.randperm(256, generator=torch.Generator().manual_seed(1))
    q = nv.MX8Tensor(torch.stack([codes, codes[order][:, order]]).to(dev()), torch.stack([scales, scales[order]]).to(dev()), 256)
    for rule in (ref4.FLOOR, ref4.CEIL):
        for sr in (nv.NVFP4_RNE, nv.NVFP4_SR):
            p = nv.mxfp4_quant_params(True, True, rule, sr, sr, 9)
            got, want = nv.mxfp8_to_mxfp4(q, p), nv.mxfp4_quantize(nv.mxfp8_dequantize(q, torch.bfloat16), p)
            assert all(equal_copies(a, b) for a, b in zip(got, want))


def test_special_scales_reach_their_block(nv):
    x = torch.randn(40, 100, device=dev())
    x[7, 40] = float("nan")
    q = nv.mxfp8_quantize(x)
    row, col = nv.mxfp8_to_mxfp4(q, nv.mxfp4_quant_params(True, True))
    bad = torch.zeros(40, 100, dtype=torch.bool, device=dev())
    bad[7, 32:64] = True
    assert torch.equal(torch.isnan(nv.mxfp8_dequantize(q)), bad)
    assert torch.equal(torch.isnan(nv.mxfp4_dequantize(row)), bad)
    cols = torch.zeros(100, 40, dtype=torch.bool, device=dev())
    cols[32:64, :32] = True
    assert torch.equal(torch.isnan(nv.mxfp4_dequantize(col)), cols)


def close(got, want, tol, what):
    """float32: within tol.  bfloat16: rounding is monotone, so between the roundings of want -+ tol."""
    if got.dtype == torch.bfloat16:
        bad = (got < (want - tol).bfloat16()) | (got > (want + tol).bfloat16()) | torch.isnan(got)
    else:
        bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}"


def gradients(g, u, dh, act, dh_error=0.0):
    """dG, dU, H in float64 and the bounds of their errors when computed in binary32 (one rounding for each
    product more than the activation's bounds hold)."""
    a, slope = ref.activation(g, act)
    ea, es = ref.activation_error(g, act)
    da, du = np.abs(dh) + dh_error, np.abs(u)
    return [(dh * u * slope, dh_error * du * (np.abs(slope) + es) + da * du * (es + 3 * ref.EPS * np.abs(slope))),
            (dh * a, dh_error * (np.abs(a) + ea) + da * (ea + 2 * ref.EPS * np.abs(a))),
            (a * u, du * (ea + 2 * ref.EPS * np.abs(a)))]


def on_gpu(pairs):
    return [(torch.from_numpy(v).to(dev()), torch.from_numpy(t + 1e-45).to(dev())) for v, t in pairs]


@pytest.mark.parametrize("act", [ref.SILU, ref.GELU])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 33), (3, 128), (5, 129), (40, 777), (300, 260), (64, 4096)])
def test_gated_backward(nv, rows, cols, act):
    print(f"mx8 backward {rows}x{cols} {act}", flush=True)
    gu = values_of((2, rows, cols), 11, torch.float32).clamp_(-60, 60)
    q = nv.mxfp8_quantize(gu)
    g, u = ref.decode(q.codes.cpu().numpy(), q.scales.cpu().numpy())[..., :cols]
    for dh_dtype in DTYPES:
        wide = values_of((rows, cols + 3), 12, dh_dtype).clamp_(-1e3, 1e3)
        dh = wide[:, 1:1 + cols]
        pairs = on_gpu(gradients(g, u, dh.double().cpu().numpy(), act))
        for dt in DTYPES:
            dgu, h = nv.mxfp8_gated_backward(dh, q, activation=act, out_dtype=dt, h=True)
            for got, pair, what in zip((dgu[:, :cols], dgu[:, cols:], h), pairs, ("dG", "dU", "H")):
                close(got, *pair, what)
            buf = torch.full((rows + 2, 2 * cols + 5), 7.0, dtype=dt, device=dev())
            hbuf = torch.full((rows + 2, cols + 3), 7.0, dtype=dt, device=dev())
            nv.mxfp8_gated_backward(dh, q, activation=act, out=buf[1:-1, 1:1 + 2 * cols], h=hbuf[1:-1, 2:2 + cols])
            assert torch.equal(buf[1:-1, 1:1 + 2 * cols], dgu) and torch.equal(hbuf[1:-1, 2:2 + cols], h)
            buf[1:-1, 1:1 + 2 * cols], hbuf[1:-1, 2:2 + cols] = 7.0, 7.0
            assert (buf == 7.0).all() and (hbuf == 7.0).all()
            only, none = nv.mxfp8_gated_backward(dh, q, activation=act, out_dtype=dt)
            assert none is None and torch.equal(only, dgu)


def test_gradients_read_every_code_and_scale(nv):
    """Far out a(g) = g and a'(g) = 1: with dH = 1 dU is the gate's value and dG the other's, whatever its code and
    scale, exactly but for results below 2^-126, which may be 0; a NaN scale makes its block NaN."""
    codes = torch.arange(256, dtype=torch.uint8, device=dev())
    codes[[127, 255]] = 0
    codes = torch.stack([torch.full((255, 256), 0x7E, dtype=torch.uint8, device=dev()), codes.repeat(255, 1)])
    scales = torch.arange(255, dtype=torch.uint8, device=dev())[:, None].repeat(1, 8)
    q = nv.MX8Tensor(codes, torch.stack([torch.full_like(scales, 127), scales]), 256)
    v = torch.from_numpy(ref.decode(codes.cpu().numpy(), q.scales.cpu().numpy())).to(dev())
    a = nv.MXTensor(torch.full((255, 64), 0x11, dtype=torch.uint8, device=dev()), torch.full((255, 4), 127, dtype=torch.uint8, device=dev()), 128)
    w = nv.MXTensor(torch.zeros(256, 64, dtype=torch.uint8, device=dev()), torch.full((256, 4), 127, dtype=torch.uint8, device=dev()), 128)
    w.codes[:, 0] = 4       # 2 x 1 / 2: dH = 1
    for nan in (False, True):
        if nan:
            q.scales[0, 3, 2], q.scales[1, 9, 5] = 255, 255
            v[:, 3, 64:96], v[1, 9, 160:192] = float("nan"), float("nan")
        for dgu, _ in (nv.mxfp8_gated_backward(torch.ones(255, 256, device=dev()), q),
                       nv.mxfp4_gated_backward(a, w, q, out_dtype=torch.float32)):
            for got, want in ((dgu[:, :256], v[1]), (dgu[:, 256:], v[0])):
                fits = want.abs() < 2.0 ** 128
                assert torch.equal(torch.isnan(got), torch.isnan(want))
                assert ((got.double() - want).abs()[fits] <= (want.abs()[fits] < 2.0 ** -126) * 2.0 ** -126).all()


@pytest.mark.parametrize("act", [ref.SILU, ref.GELU])
def test_gradients_far_out(nv, act):
    """Gates at which the exponential overflows or vanishes: finite gradients, 0 or 1 in the limit."""
    g = torch.tensor([-448.0, -200, -120, -88, 88, 120, 200, 448], device=dev()).repeat(1, 4)
    q = nv.mxfp8_quantize(torch.stack([g, torch.ones_like(g)]))
    v = nv.mxfp8_dequantize(q).double().cpu().numpy()
    dgu, h = nv.mxfp8_gated_backward(torch.ones_like(g), q, activation=act, h=True)
    assert torch.isfinite(dgu).all() and torch.isfinite(h).all()
    pairs = on_gpu(gradients(v[0], v[1], np.ones(v[0].shape), act))
    for got, pair, what in zip((dgu[:, :32], dgu[:, 32:], h), pairs, ("dG", "dU", "H")):
        close(got, *pair, what)


@pytest.mark.parametrize("act", [ref.SILU, ref.GELU])
def test_gradients_at_the_ends_of_the_range(nv, act):
    """From 2^9 on a(g) = g and a'(g) = 1, or both 0 (binary32 leaves nothing else), up to the largest g there is."""
    g = torch.tensor([s * v for v in (512.0, 1e6, 1.5e19, 2e19, 1e30, 3e38) for s in (1, -1)], device=dev()).repeat_interleave(32)[None]
    u = torch.full_like(g, 1.5)
    q = nv.mxfp8_quantize(torch.stack([g, u]))
    v = nv.mxfp8_dequantize(q)
    a = nv.MXTensor(torch.full((1, 64), 0x11, dtype=torch.uint8, device=dev()), torch.full((1, 4), 127, dtype=torch.uint8, device=dev()), 128)
    w = nv.MXTensor(torch.zeros(g.numel(), 64, dtype=torch.uint8, device=dev()), torch.full((g.numel(), 4), 127, dtype=torch.uint8, device=dev()), 128)
    w.codes[:, 0] = 4       # 2 x 1 / 2: dH = 1
    for dgu, h in (nv.mxfp8_gated_backward(torch.ones_like(g), q, activation=act, out_dtype=torch.float32, h=True),
                   nv.mxfp4_gated_backward(a, w, q, activation=act, out_dtype=torch.float32, h=True)):
        n = g.numel()
        assert torch.equal(dgu[:, :n], torch.where(g > 0, 1.5, 0.0))
        assert torch.equal(dgu[:, n:], torch.where(g > 0, v[0], 0.0))
        assert torch.equal(h, torch.where(g > 0, 1.5 * v[0], 0.0))      # an infinity where that leaves the range
