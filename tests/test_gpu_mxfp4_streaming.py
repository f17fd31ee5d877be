"""The MXFP4 kernels' variants for large data, which go past the caches: float32 results from 256 MiB
on (gradients of groups from 128 MiB), inputs of the quantizer from 128 MiB on."""
import numpy as np
import pytest
import torch

import mxfp4_reference as ref
from gpu_util import GEMM_TOL, dev
from test_gpu_mxfp4_gemm import copy_of, product, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load_library()
    return nv


def check(c, want, absdot, what):
    """|error| <= GEMM_TOL * sum |a b|: products are exact, only the FP32 accumulation rounds."""
    bad = ~((c.double() - want).abs() <= GEMM_TOL * absdot)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"


def framed(shape):
    """A float32 matrix inside a larger one of NaN."""
    buf = torch.full((shape[0] + 2, shape[1] + 7), float("nan"), device=dev())
    return buf, buf[1:-1, 3:3 + shape[1]]


def untouched(buf, inner):
    inner.fill_(float("nan"))
    return bool(torch.isnan(buf).all())


# in tiles of 256 x 256: 36 x 30 of them, K of less than one stage and of several; and of 128 x 128 (one
# column of tiles, half of which a larger one would waste)
@pytest.mark.parametrize("M,N,K", [(9001, 7479, 100), (8193, 8200, 1500), (600001, 120, 64), (120, 570001, 300)])
def test_dense(nv, M, N, K):
    assert M * N * 4 > 256 << 20
    print(f"dense {M}x{N}x{K}", flush=True)
    a, b = copy_of(nv, (M,), K, 51), copy_of(nv, (N,), K, 52)
    buf, out = framed((M, N))
    nv.mxfp4_gemm(a, b, out=out)
    check(out, *product(values(a), values(b)), "dense")
    assert untouched(buf, out)


def some_offsets(rows, groups, seed, tail):
    """Ends of the groups at random, every third group empty, `tail` rows in none."""
    off = [0, *np.sort(np.random.RandomState(seed).randint(0, rows - tail + 1, groups - 1)).tolist(), rows - tail]
    for g in range(1, groups, 3):
        off[g] = off[g - 1]
    return off


@pytest.mark.parametrize("M,N,K,G", [(9000, 7777, 200, 5), (34000, 2100, 130, 70), (560000, 123, 200, 100)])
def test_grouped_rows(nv, M, N, K, G):
    assert M * N * 4 > 256 << 20
    print(f"grouped rows {M}x{N}x{K} {G}", flush=True)
    off = some_offsets(M, G, 53, 300)
    a, b = copy_of(nv, (M,), K, 54), copy_of(nv, (G, N), K, 55)
    buf, out = framed((M, N))
    nv.mxfp4_gemm_grouped(a, b, torch.tensor(off, dtype=torch.int32, device=dev()), out=out)
    va, vb = values(a), values(b)
    for g, (i, j) in enumerate(ref.spans(off, M)):
        if j > i:
            check(out[i:j], *product(va[i:j], vb[g]), f"group {g}")
    assert (out[off[-1]:] == 0).all()
    assert untouched(buf, out)


@pytest.mark.parametrize("rows,N,K,G", [(700, 1500, 2600, 9), (3000, 100, 3000, 120), (2500, 2049, 2300, 8)])
def test_grouped_wgrad(nv, rows, N, K, G):
    assert G * N * K * 4 > 128 << 20
    print(f"wgrad {rows} rows {G}x{N}x{K}", flush=True)
    off = some_offsets(rows, G, 56, 20)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    gen = torch.Generator(device=dev()).manual_seed(57)
    p = nv.mxfp4_quant_params(False, True, ref.CEIL)
    dyc, xc = (nv.mxfp4_quantize(torch.randn(rows, n, generator=gen, device=dev()), p, offsets=offsets)[1] for n in (N, K))
    dyv, xv = (nv.mxfp4_dequantize(q, offsets=offsets).double() for q in (dyc, xc))
    c = nv.mxfp4_gemm_grouped_wgrad(dyc, xc, offsets, out=torch.full((G, N, K), float("nan"), device=dev()))
    for g, (i, j) in enumerate(ref.spans(off, rows)):
        if j > i:
            check(c[g], *product(dyv[:, i:j], xv[:, i:j]), f"group {g}")
        else:
            assert (c[g] == 0).all()


def wide_input(R, C, dtype, seed):
    """A view of R x C with an odd pitch and start, values of many sizes, some zeros and a NaN."""
    gen = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randn(R, C + 5, generator=gen, device=dev())
    x *= torch.exp2(torch.randint(-6, 7, x.shape, generator=gen, device=dev()).float())
    x[torch.rand(x.shape, generator=gen, device=dev()) < 0.02] = 0
    x = x.to(dtype)[:, 3:3 + C]
    x[R // 2, C // 3] = float("nan")
    return x


LARGE = [(8209, 8401, torch.bfloat16), (4101, 8399, torch.float32)]


@pytest.mark.parametrize("R,C,dtype", LARGE)
@pytest.mark.parametrize("rounding", [0, 1])
def test_quantize(nv, R, C, dtype, rounding):
    """Sampled rows and columns against the reference, and (to nearest) all codes against those of parts
    that are small enough to be read through the caches."""
    x = wide_input(R, C, dtype, 58)
    assert R * C * x.element_size() >= 128 << 20
    print(f"quantize {R}x{C} {dtype} {rounding}", flush=True)
    seed = 0xFEDCBA9876543210
    row, col = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(True, True, ref.CEIL, rounding, rounding, seed))
    r = np.random.RandomState(59)
    for q, v, copy in ((row, x, 0), (col, x.t(), 1)):
        n, k = v.shape
        at = np.unique(np.r_[0, n - 1, (R // 2, C // 3)[copy], r.randint(0, n, 40)])
        bits = np.concatenate([row_bits(i, ref.pad128(k), copy, seed) for i in at]) if rounding else None
        nib, sc = ref.quantize_rows(v[torch.from_numpy(at).to(dev())].float().cpu().numpy().astype(np.float64), ref.CEIL, bits)
        pick = torch.from_numpy(at).to(dev())
        assert np.array_equal(q.scales[pick].cpu().numpy(), sc)
        assert np.array_equal(ref.unpack(q.codes[pick].cpu().numpy()), nib)
    if rounding:
        return
    for i in range(0, R, 2048):
        part = x[i:i + 2048]
        pr, pc = nv.mxfp4_quantize(part, nv.mxfp4_quant_params(True, True, ref.CEIL))
        assert torch.equal(pr.codes, row.codes[i:i + 2048]) and torch.equal(pr.scales, row.scales[i:i + 2048])
        kp = ref.pad128(part.shape[0])
        assert torch.equal(pc.codes, col.codes[:, i // 2:(i + kp) // 2])
        assert torch.equal(pc.scales, col.scales[:, i // 32:(i + kp) // 32])


def row_bits(i, kp, copy, seed):
    """ref.sr_bits of row i alone: elements i kp .. i kp + kp - 1 of the copy."""
    blocks = np.arange(i * kp // 8, (i + 1) * kp // 8, dtype=np.uint64)
    ctr = np.stack([blocks & np.uint64(0xFFFFFFFF), blocks >> np.uint64(32), np.full_like(blocks, copy),
                    np.full_like(blocks, 0x4D585352)], 1)
    w = ref.philox_words(ctr.astype(np.uint32), seed)
    return np.stack([w & 0xFFFF, w >> 16], -1).reshape(1, kp).astype(np.int64)


@pytest.mark.parametrize("R,C,dtype", LARGE)
def test_quantize_groups(nv, R, C, dtype):
    x = wide_input(R, C, dtype, 60)
    off = some_offsets(R, 90, 61, 200)
    print(f"quantize groups {R}x{C} {dtype}", flush=True)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    _, col = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(False, True), offsets=offsets)
    at = np.unique(np.r_[0, C - 1, C // 3, np.random.RandomState(62).randint(0, C, 40)])
    pick = torch.from_numpy(at).to(dev())
    nib, sc = ref.quantize_grouped_cols(x[:, pick].float().cpu().numpy().astype(np.float64), off, col.codes.shape[1] * 2)
    used = nib.shape[1]
    assert np.array_equal(col.scales[pick].cpu().numpy()[:, :used // 32], sc)
    assert np.array_equal(ref.unpack(col.codes[pick].cpu().numpy())[:, :used], nib)


def test_row_bits_are_the_references():
    full = ref.sr_bits(5, 256, 1, 77)
    assert np.array_equal(np.concatenate([row_bits(i, 256, 1, 77) for i in range(5)]), full)
