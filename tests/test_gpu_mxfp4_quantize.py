"""MXFP4 quantization on the GPU against the plain 64-bit reference, bit for bit: E8M0 scale
codes, E2M1 nibbles (nearest even and stochastic) and padding of both copies, over odd sizes,
strides, alignments, stacks, groups and special values; and the decode's exact values."""
import numpy as np
import pytest
import torch

import mxfp4_reference as ref
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load_library()
    return nv


def make(rows, cols, dtype, seed, spread=8):
    """Normal values times a power of two that varies from element to element."""
    r = np.random.RandomState(seed)
    v = r.randn(rows, cols) * 2.0 ** r.randint(-spread, spread, (rows, cols))
    v[r.rand(rows, cols) < 0.02] = 0.0
    return torch.from_numpy(v.astype(np.float32)).to(dtype)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check_copy(q, want, what, used=None):
    nib, sc = want
    codes, scales = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    if used is not None:
        codes, scales = codes[:, :used // 2], scales[:, :used // 32]
    bad = np.argwhere(scales != sc)
    assert bad.size == 0, f"{what}: {len(bad)} scales, first {bad[0]}: {scales[tuple(bad[0])]} vs {sc[tuple(bad[0])]}"
    got = ref.unpack(codes)
    bad = np.argwhere(got != nib)
    assert bad.size == 0, f"{what}: {len(bad)} codes, first {bad[0]}: {got[tuple(bad[0])]} vs {nib[tuple(bad[0])]}"


SIZES = [(1, 1), (1, 32), (2, 31), (3, 33), (31, 7), (32, 128), (33, 129), (128, 64), (127, 257),
         (129, 1000), (257, 384), (1, 4096), (640, 65)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rule", [ref.FLOOR, ref.CEIL])
@pytest.mark.parametrize("rounding", [0, 1])
def test_both_copies(nv, dtype, rule, rounding):
    for i, (R, C) in enumerate(SIZES):
        print(f"both copies {R}x{C} {dtype} rule {rule} rounding {rounding}", flush=True)
        x = make(R, C, dtype, 10 + i)
        seed = 0x123456789ABCDEF + i
        p = nv.mxfp4_quant_params(True, True, rule, rounding, rounding, seed)
        row, col = nv.mxfp4_quantize(x.to(dev()), p)
        v = f64(x)
        bits = lambda n, k, c: ref.sr_bits(n, ref.pad128(k), c, seed) if rounding else None
        check_copy(row, ref.quantize_rows(v, rule, bits(R, C, 0)), f"row {R}x{C}")
        check_copy(col, ref.quantize_rows(v.T, rule, bits(C, R, 1)), f"col {R}x{C}")
        assert row.shape == (R, C) and col.shape == (C, R)
        # one copy alone, and different roundings, give the same
        one, none = nv.mxfp4_quantize(x.to(dev()), nv.mxfp4_quant_params(True, False, rule, rounding, 0, seed))
        assert none is None and torch.equal(one.codes, row.codes) and torch.equal(one.scales, row.scales)
        none, one = nv.mxfp4_quantize(x.to(dev()), nv.mxfp4_quant_params(False, True, rule, 1 - rounding,
                                                                         rounding, seed))
        assert none is None and torch.equal(one.codes, col.codes) and torch.equal(one.scales, col.scales)
        mixed = nv.mxfp4_quantize(x.to(dev()), nv.mxfp4_quant_params(True, True, rule, rounding,
                                                                     1 - rounding, seed))
        assert torch.equal(mixed[0].codes, row.codes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("first,pitch", [(0, 0), (1, 0), (0, 3), (3, 8), (8, 64)])
def test_strided_and_unaligned_views(nv, dtype, first, pitch):
    R, C = 150, 203
    wide = make(R, C + first + pitch, dtype, 5).to(dev())
    x = wide[:, first:first + C]
    row, col = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(True, True))
    check_copy(row, ref.quantize_rows(f64(x)), "row")
    check_copy(col, ref.quantize_rows(f64(x).T), "col")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_stack_of_matrices(nv, dtype):
    big = make(3 * 140, 150, dtype, 6).reshape(3, 140, 150).to(dev())
    for x in (big, big[:, 3:133, 5:70], big[::2], big[1:2, :1]):
        row, col = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(True, True, ref.CEIL, 0, 1, 77))
        B, R, C = x.shape
        bits = ref.sr_bits(B * C, ref.pad128(R), 1, 77).reshape(B, C, -1)
        for b in range(B):
            v = f64(x[b])
            check_copy(nv.MXTensor(row.codes[b], row.scales[b], C), ref.quantize_rows(v, ref.CEIL), "row")
            check_copy(nv.MXTensor(col.codes[b], col.scales[b], R), ref.quantize_rows(v.T, ref.CEIL, bits[b]),
                       "col")
        got = nv.mxfp4_dequantize(row)
        assert got.shape == x.shape
        want = ref.decode(*ref.quantize_rows(f64(x).reshape(-1, C), ref.CEIL))[:, :C].reshape(B, R, C)
        assert np.array_equal(f64(got), want)


GROUPS = [
    (300, [0, 300]),
    (300, [0, 0, 1, 129, 129, 257, 300]),
    (1000, [0, 128, 256, 999, 1000]),
    (40, [0] + sorted(np.random.RandomState(0).randint(0, 41, 70).tolist()) + [40]),   # more than 64 groups
    (700, [0] + sorted(np.random.RandomState(1).randint(0, 600, 130).tolist())),       # a tail in no group
    (200, [0, 0, 0]),                                                                  # no row in a group
    (300, [0, 200, 100, 5000, -3, 300]),     # clamped: 0-200, empty, 200-300, empty, empty
    (300, [7, 100, 300]),                    # the first entry is read as 0
]


@pytest.mark.parametrize("case", range(len(GROUPS)))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped_columns(nv, case, dtype):
    rows, off = GROUPS[case]
    C = 77
    print(f"groups {case} {dtype}", flush=True)
    x = make(rows, C, dtype, 20 + case)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    for rounding in (0, 1):
        p = nv.mxfp4_quant_params(True, True, ref.CEIL, 0, rounding, 99)
        row, col = nv.mxfp4_quantize(x.to(dev()), p, offsets=offsets)
        check_copy(row, ref.quantize_rows(f64(x), ref.CEIL), "row")
        kp = col.codes.shape[1] * 2
        bits = ref.sr_bits(C, kp, 1, 99) if rounding else None
        want = ref.quantize_grouped_cols(f64(x), off, kp, ref.CEIL, bits)
        used = want[0].shape[1]
        assert used <= kp
        check_copy(col, want, "col", used)
    pos, inside, _ = ref.grouped_positions(off, rows)
    value = np.zeros((C, rows))
    value[:, inside] = ref.decode(*want)[:, pos[inside]]
    for od in (torch.float32, torch.bfloat16):
        got = nv.mxfp4_dequantize(col, od, offsets=offsets)
        assert np.array_equal(f64(got), value)


def test_special_values(nv):
    """Zero blocks, signed zeros, infinities and NaN, subnormals, the largest values, ties."""
    big, tiny = np.float32(3.4028235e38), np.float32(1e-45)
    rows = [np.zeros(32), np.full(32, -0.0), np.r_[np.inf, np.ones(31)], np.r_[np.nan, np.ones(31)],
            np.r_[-np.inf, np.nan, np.ones(30)], np.full(32, tiny), np.r_[tiny, -1e-39, 2e-39, np.zeros(29)],
            np.r_[big, -big, 1e38, 2e38, np.zeros(28)], np.r_[1.1754944e-38, 5e-39, np.zeros(30)],
            np.r_[6.0, np.arange(31) / 4 - 3.75], np.r_[4.0, np.arange(31) / 4 - 3.75],
            np.r_[7.99, np.arange(31) / 4 - 3.75], np.r_[6.01, np.arange(31) / 8], np.r_[-5, -7, 3.5, 2.5, np.ones(28)],
            np.r_[2.0 ** -125, np.zeros(31)], np.r_[2.0 ** -124 * 1.75, np.zeros(31)]]
    x = np.stack(rows).astype(np.float32)
    x = np.concatenate([x, x[::-1]], 1)
    for dtype in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(x).to(dtype)
        v = f64(t)
        for rule in (ref.FLOOR, ref.CEIL):
            row, col = nv.mxfp4_quantize(t.to(dev()), nv.mxfp4_quant_params(True, True, rule))
            want = ref.quantize_rows(v, rule)
            check_copy(row, want, f"row {dtype} {rule}")
            check_copy(col, ref.quantize_rows(v.T, rule), f"col {dtype} {rule}")
            value = ref.decode(*want)[:, :x.shape[1]]
            for od in (torch.float32, torch.bfloat16):
                got = f64(nv.mxfp4_dequantize(row, od))
                assert np.array_equal(got, value.astype(np.float32).astype(np.float64), equal_nan=True)
                assert np.array_equal(np.signbit(got)[value == 0], np.signbit(value)[value == 0])


def test_every_bf16_value(nv):
    """Each bfloat16 alone in a block, and beside amax 1.5 (every rounding of E2M1)."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros(65536, 64, dtype=torch.bfloat16)
    x[:, 5] = every
    x[:, 32] = 1.5
    x[:, 40] = every
    for rule in (ref.FLOOR, ref.CEIL):
        row, _ = nv.mxfp4_quantize(x.to(dev()), nv.mxfp4_quant_params(True, False, rule))
        check_copy(row, ref.quantize_rows(f64(x), rule), f"rule {rule}")


def test_dequantize_into_views_and_every_code(nv):
    r = np.random.RandomState(3)
    n, k = 37, 300
    codes = r.randint(0, 256, (n, 192)).astype(np.uint8)
    scales = r.randint(0, 256, (n, 12)).astype(np.uint8)
    q = nv.MXTensor(torch.from_numpy(codes).to(dev()), torch.from_numpy(scales).to(dev()), k)
    with np.errstate(over="ignore"):
        value = ref.decode(ref.unpack(codes), scales)[:, :k].astype(np.float32)
    assert np.array_equal(nv.mxfp4_dequantize(q).cpu().numpy(), value, equal_nan=True)
    for od in (torch.float32, torch.bfloat16):
        buf = torch.full((n + 2, k + 9), 7.0, dtype=od, device=dev())
        nv.mxfp4_dequantize(q, out=buf[1:-1, 3:3 + k])
        want = torch.from_numpy(value).to(od)
        assert torch.equal(torch.nan_to_num(buf[1:-1, 3:3 + k].cpu().float()), torch.nan_to_num(want.float()))
        buf[1:-1, 3:3 + k] = 7.0
        assert (buf == 7.0).all()


def test_stochastic_rounding_is_unbiased(nv):
    """Mean over 4096 draws of a value between two grid points; standard error 0.5 / 64 of the
    spacing, five of them allowed."""
    x = torch.full((4096, 32), 0.3, device=dev())
    x[:, 0] = 6.0
    x[:, 1] = 4.9
    row, _ = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(True, False, ref.CEIL, 1, 0, 5))
    v = nv.mxfp4_dequantize(row).double()
    assert abs(v[:, 1].mean().item() - 4.9) < 5 * 2 * 0.5 / 64
    assert abs(v[:, 2:].mean().item() - 0.3) < 5 * 0.5 * 0.5 / 64 / 30 ** 0.5


def test_large_offsets(nv):
    """Elements past 2^31 of a wide view: the last rows of a matrix with a 2^24-element pitch."""
    R, C, ld = 140, 40, 1 << 24
    buf = torch.empty(R * ld, dtype=torch.bfloat16, device=dev())
    x = buf.view(R, ld)[:, ld - C:]
    x.copy_(make(R, C, torch.bfloat16, 8))
    row, col = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(True, True))
    check_copy(row, ref.quantize_rows(f64(x)), "row")
    check_copy(col, ref.quantize_rows(f64(x).T), "col")


def test_empty(nv):
    for shape in [(0, 5), (5, 0), (0, 0), (0, 4, 4)]:
        row, col = nv.mxfp4_quantize(torch.empty(shape, device=dev()), nv.mxfp4_quant_params(True, True))
        assert row.shape == shape and nv.mxfp4_dequantize(row).shape == shape
        assert col.shape == (*shape[:-2], shape[-1], shape[-2])


def test_refusals(nv):
    x = torch.zeros(8, 64, device=dev())
    p = nv.mxfp4_quant_params(True, True)
    off = torch.tensor([0, 8], dtype=torch.int32, device=dev())
    for bad in (x.half(), x.double(), x.cpu(), x.t(), x[0], x.view(1, 1, 8, 64)):
        with pytest.raises(nv.Nvfp4Error):
            nv.mxfp4_quantize(bad, p)
    for kw in ({"offsets": off.long()}, {"offsets": off.cpu()}, {"offsets": off[:1]}, {"offsets": off.view(1, 2)},
               {"row_out": nv.MXTensor.empty(8, 32, dev())}, {"col_out": nv.MXTensor.empty(64, 8, dev(), 2)},
               {"row_out": nv.MXTensor.empty(7, 64, dev())}):
        with pytest.raises(nv.Nvfp4Error):
            nv.mxfp4_quantize(x, p, **kw)
    with pytest.raises(nv.Nvfp4Error):
        nv.mxfp4_quantize(x.view(2, 4, 64), p, offsets=off)
    for bad in (nv.mxfp4_quant_params(False, False), nv.mxfp4_quant_params(True, False, 2),
                nv.mxfp4_quant_params(True, False, 0, 2), nv.mxfp4_quant_params(True, False, 0, 0, -1)):
        with pytest.raises(nv.Nvfp4Error):
            nv.mxfp4_quantize(x, bad)
    row, col = nv.mxfp4_quantize(x, p, offsets=off)
    with pytest.raises(nv.Nvfp4Error):
        nv.mxfp4_dequantize(col)                      # needs its offsets
    with pytest.raises(nv.Nvfp4Error):
        nv.mxfp4_dequantize(row, offsets=off)
    with pytest.raises(nv.Nvfp4Error):
        nv.mxfp4_dequantize(row, torch.float16)
    with pytest.raises(nv.Nvfp4Error):
        nv.mxfp4_dequantize(row, out=torch.empty(8, 63, device=dev()))
