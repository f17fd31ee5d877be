"""MXFP4 products on the GPU against float64 products of the decoded operands: dense, grouped
rows, ragged K, and the one-call layer, over sizes around every tile edge."""
import numpy as np
import pytest
import torch

import mxfp4_reference as ref
from gpu_util import GEMM_TOL, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load_library()
    return nv


def copy_of(nv, lead, k, seed, spread=6):
    """A random copy: any codes up to k, scales 2^-spread .. 2^spread, zero padding."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    kp = ref.pad128(k)
    nib = torch.randint(0, 16, (*lead, kp), generator=g, device=dev(), dtype=torch.uint8)
    nib[..., k:] = 0
    sc = torch.randint(127 - spread, 128 + spread, (*lead, kp // 32), generator=g, device=dev()).to(torch.uint8)
    sc[..., -(-k // 32):] = 0
    return nv.MXTensor(nib[..., 0::2] | (nib[..., 1::2] << 4), sc, k)


def values(q):
    """Decoded values [.., kp] in float64, on the GPU, by the table of E2M1."""
    table = torch.tensor(ref.VALUES, device=q.codes.device)
    v = torch.stack([table[(q.codes & 15).long()], table[(q.codes >> 4).long()]], -1).flatten(-2)
    s = ((q.scales.long() - 127 + 1023) << 52).view(torch.float64)   # 2^(code - 127)
    return v * s.repeat_interleave(32, -1)


def check(c, want, absdot, what):
    """float32: |error| <= GEMM_TOL * sum |a b| (products are exact; only the FP32 accumulation
    rounds).  bfloat16: one rounding of such a value; rounding is monotone, so C lies between
    the roundings of the two ends."""
    err, tol = (c.double() - want).abs(), GEMM_TOL * absdot
    if c.dtype == torch.bfloat16:
        bad = (c < (want - tol).bfloat16()) | (c > (want + tol).bfloat16()) | torch.isnan(c)
    else:
        bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {(err / absdot.clamp(min=1e-300)).max().item():.3g}"


def product(a, b):
    return a @ b.transpose(-1, -2).contiguous(), a.abs() @ b.abs().transpose(-1, -2).contiguous()


DTYPES = [(torch.float32, "f32"), (torch.bfloat16, "bf16")]
DENSE = [(1, 1, 1), (1, 4096, 128), (1, 33, 4096), (2, 300, 2080), (7, 129, 31), (16, 16, 32), (17, 1000, 1000),
         (31, 65, 257), (32, 512, 512), (33, 257, 640), (64, 2049, 384), (65, 64, 129), (100, 100, 100),
         (128, 128, 256), (129, 127, 384), (200, 700, 1500), (255, 256, 512), (256, 255, 1024), (257, 511, 130),
         (300, 1, 700), (513, 513, 2500), (1024, 2048, 896), (2000, 130, 4097), (2304, 2560, 1152)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(nv, M, N, K):
    print(f"dense {M}x{N}x{K}", flush=True)
    a, b = copy_of(nv, (M,), K, 1), copy_of(nv, (N,), K, 2)
    want, absdot = product(values(a), values(b))
    for dt, name in DTYPES:
        c = nv.mxfp4_gemm(a, b, out_dtype=dt)
        assert c.dtype == dt
        check(c, want, absdot, f"dense {name}")
        # a view with a wider pitch: the same values, nothing written beside them
        buf = torch.full((M + 2, N + 5), 3.0, dtype=dt, device=dev())
        nv.mxfp4_gemm(a, b, out=buf[1:-1, 2:2 + N])
        assert torch.equal(buf[1:-1, 2:2 + N], c)
        buf[1:-1, 2:2 + N] = 3.0
        assert (buf == 3.0).all()


@pytest.mark.parametrize("M,N,K", [(6144, 5000, 640), (6100, 4990, 130), (5000, 4100, 1500), (6144, 5120, 257)])
def test_dense_more_tiles_than_compute_units(nv, M, N, K):
    """Workgroups that go through several large tiles, whole ones and ones cut at C's edges."""
    test_dense(nv, M, N, K)


def test_scales_far_apart_and_nan(nv):
    """Block scales from 2^-60 to 2^60; a NaN scale reaches exactly its row or column."""
    a, b = copy_of(nv, (70,), 500, 3, spread=60), copy_of(nv, (90,), 500, 4, spread=60)
    want, absdot = product(values(a), values(b))
    check(nv.mxfp4_gemm(a, b), want, absdot, "far apart f32")
    a, b = copy_of(nv, (70,), 500, 3), copy_of(nv, (90,), 500, 4)
    want, absdot = product(values(a), values(b))
    a.scales[7, 3] = 255
    b.scales[80, 15] = 255
    c = nv.mxfp4_gemm(a, b)
    nan = torch.zeros(70, 90, dtype=torch.bool, device=dev())
    nan[7] = True
    nan[:, 80] = True
    assert torch.equal(torch.isnan(c), nan)
    check(c[~nan], want[~nan], absdot[~nan], "beside NaN f32")


@pytest.mark.parametrize("M", [7, 14, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_inputs_with_nan_and_inf(nv, M, dtype):
    """A token with a NaN or an infinity gives NaN in its own row of Y only."""
    x = torch.randn(M, 300, device=dev()).to(dtype)
    x[3, 200], x[6, 0] = float("nan"), float("inf")
    w = nv.mxfp4_quantize(torch.randn(50, 300, device=dev()), nv.mxfp4_quant_params())[0]
    off = torch.tensor([0, 5, M], dtype=torch.int32, device=dev())
    stack = nv.MXTensor(torch.stack([w.codes] * 2), torch.stack([w.scales] * 2), 300)
    for y in (nv.mxfp4_linear(x, w), nv.mxfp4_linear(x, stack, offsets=off)):
        assert torch.isnan(y).any(1).nonzero().flatten().tolist() == [3, 6]
        assert torch.isnan(y[[3, 6]]).all()


def spread_offsets(rows, groups, seed, tail=0):
    cut = np.sort(np.random.RandomState(seed).randint(0, rows - tail + 1, groups - 1)) if groups > 1 else []
    return [0, *[int(c) for c in cut], rows - tail]


GROUPED = [(1, 3, 40, 96, [0, 0, 1, 1]), (24, 8, 300, 500, spread_offsets(24, 8, 0)),
           (100, 3, 257, 130, [0, 33, 33, 100]), (600, 5, 256, 384, [0, 256, 257, 300, 600, 600]),
           (900, 70, 96, 160, spread_offsets(900, 70, 1)), (1500, 4, 520, 1000, spread_offsets(1500, 4, 2, tail=300)),
           (64, 2, 65, 64, [0, 0, 0]), (300, 3, 100, 64, [5, 900, 2, 300]), (4000, 6, 300, 700, spread_offsets(4000, 6, 4))]


def many_offsets(rows, groups, seed, tail=0):
    """Every third group empty."""
    off = spread_offsets(rows, groups, seed, tail)
    for g in range(1, groups, 3):
        off[g] = off[g - 1]
    return off


# more large tiles than compute units: several per workgroup, some without anything to multiply
GROUPED_MANY = [(6000, 5, 4600, 300, [0, 2000, 2000, 2600, 2601, 5500]), (20000, 70, 2100, 200, many_offsets(20000, 70, 7, 100)),
                (6144, 4, 4608, 512, [0, 1536, 3072, 4608, 6144])]
WGRAD_MANY = [(3000, 9, 1500, 1536, [0, 0, 100, 1300, 1300, 1428, 2000, 2001, 2500, 3000]),
              (9000, 120, 500, 512, many_offsets(9000, 120, 8, 50))]


@pytest.mark.parametrize("case", range(len(GROUPED) + len(GROUPED_MANY)))
def test_grouped_rows(nv, case):
    M, G, N, K, off = (GROUPED + GROUPED_MANY)[case]
    print(f"grouped rows {case}", flush=True)
    a, b = copy_of(nv, (M,), K, 5), copy_of(nv, (G, N), K, 6)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    va, vb = values(a), values(b)
    want, absdot = torch.zeros(M, N, device=dev(), dtype=torch.float64), torch.zeros(M, N, device=dev(), dtype=torch.float64)
    for g, (i, j) in enumerate(ref.spans(off, M)):
        if j > i:
            want[i:j], absdot[i:j] = product(va[i:j], vb[g])
    for dt, name in DTYPES:
        buf = torch.full((M + 2, N + 3), float("nan"), dtype=dt, device=dev())
        c = nv.mxfp4_gemm_grouped(a, b, offsets, out=buf[1:-1, :N])
        check(c, want, absdot, f"grouped {name}")
        assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all() and torch.isnan(buf[:, N:]).all()


@pytest.mark.parametrize("case", range(len(GROUPED) + len(WGRAD_MANY)))
def test_grouped_wgrad(nv, case):
    rows, G, N, K, off = (GROUPED + WGRAD_MANY)[case]
    print(f"grouped wgrad {case}", flush=True)
    g = torch.Generator(device=dev()).manual_seed(case)
    x = torch.randn(rows, K, generator=g, device=dev())
    dy = torch.randn(rows, N, generator=g, device=dev())
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    p = nv.mxfp4_quant_params(False, True, ref.CEIL)
    xc, dyc = nv.mxfp4_quantize(x, p, offsets=offsets)[1], nv.mxfp4_quantize(dy, p, offsets=offsets)[1]
    xv = nv.mxfp4_dequantize(xc, offsets=offsets).double()
    dyv = nv.mxfp4_dequantize(dyc, offsets=offsets).double()
    # positions past the groups hold whatever the buffer held: NaN scales must not matter
    used = ref.grouped_positions(off, rows)[2]
    for q in (xc, dyc):
        q.codes[:, used // 2:] = 0x77
        q.scales[:, used // 32:] = 255
    for dt, name in DTYPES:
        c = nv.mxfp4_gemm_grouped_wgrad(dyc, xc, offsets, out_dtype=dt)
        assert c.shape == (G, N, K)
        for e, (i, j) in enumerate(ref.spans(off, rows)):
            if j == i:
                assert (c[e] == 0).all()
            else:
                check(c[e], *product(dyv[:, i:j], xv[:, i:j]), f"wgrad {name}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rule", [ref.FLOOR, ref.CEIL])
def test_linear_is_quantize_then_product(nv, dtype, rule):
    for M, N, K in [(1, 5000, 1024), (1, 31, 70), (3, 1025, 3000), (16, 640, 513), (33, 700, 260), (70, 257, 128),
                    (300, 515, 777), (2100, 300, 512)]:
        print(f"linear {M}x{N}x{K} {dtype} {rule}", flush=True)
        x = torch.randn(M, K + 3, device=dev()).to(dtype)[:, 1:1 + K]
        w = copy_of(nv, (N,), K, 7)
        q = ref.quantize_rows(x.float().cpu().numpy().astype(np.float64), rule)
        want, absdot = product(torch.from_numpy(ref.decode(*q)).to(dev()), values(w))
        for dt, name in DTYPES:
            check(nv.mxfp4_linear(x, w, scale_rule=rule, out_dtype=dt), want, absdot, f"linear {name}")
        assert nv.mxfp4_linear(x, w).dtype == dtype


@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_linear(nv, case):
    M, G, N, K, off = GROUPED[case]
    print(f"grouped linear {case}", flush=True)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(M, K, device=dev()).to(dtype)
        w = copy_of(nv, (G, N), K, 8)
        q = nv.mxfp4_quantize(x, nv.mxfp4_quant_params())[0]
        qv, wv = values(q), values(w)
        for dt, name in DTYPES:
            c = nv.mxfp4_linear(x, w, offsets=offsets, out_dtype=dt)
            inside = torch.zeros(M, dtype=torch.bool, device=dev())
            for g, (i, j) in enumerate(ref.spans(off, M)):
                inside[i:j] = True
                if j > i:
                    check(c[i:j], *product(qv[i:j], wv[g]), f"grouped linear {name}")
            assert (c[~inside] == 0).all()


# few rows: K past 64 KiB of LDS, past all of it, rows that fill a unit or not, both splits
FEW = [(16, 40, 9000, None), (8, 300, 9000, None), (16, 33, 20001, None), (1, 50, 20001, None), (12, 4100, 2048, None),
       (16, 2048, 1024, None), (3, 7300, 96, None), (4, 1030, 2048, [0, 1, 2, 3, 4]), (16, 70, 9000, [0, 0, 16] + [16] * 14),
       (30, 700, 260, [0, 3, 3, 4, 20] + [20] * 15 + [29]), (17, 513, 384, [1, 17])]


@pytest.mark.parametrize("case", range(len(FEW)))
def test_few_rows(nv, case):
    M, N, K, off = FEW[case]
    print(f"few rows {case}", flush=True)
    lead = (N,) if off is None else (len(off) - 1, N)
    offsets = None if off is None else torch.tensor(off, dtype=torch.int32, device=dev())
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(M, K, device=dev()).to(dtype)
        w = copy_of(nv, lead, K, 21)
        q = nv.mxfp4_quantize(x, nv.mxfp4_quant_params())[0]
        qv, wv = values(q), values(w)
        for dt, name in DTYPES:
            got = [nv.mxfp4_linear(x, w, offsets=offsets, out_dtype=dt)]
            got.append(nv.mxfp4_gemm(q, w, out_dtype=dt) if off is None else nv.mxfp4_gemm_grouped(q, w, offsets, out_dtype=dt))
            for c in got:
                if off is None:
                    check(c, *product(qv, wv), f"few {name}")
                    continue
                inside = torch.zeros(M, dtype=torch.bool, device=dev())
                for g, (i, j) in enumerate(ref.spans(off, M)):
                    inside[i:j] = True
                    if j > i:
                        check(c[i:j], *product(qv[i:j], wv[g]), f"few {name}")
                assert (c[~inside] == 0).all()


# the few-row kernel's other tiles: (M, N, K, offsets)
SMALL = [(20, 2000, 512, None), (24, 4000, 256, None), (130, 3000, 96, None), (40, 33, 9000, None), (40, 33, 10000, None),
         (100, 1500, 10000, None), (1000, 250, 1030, None), (8000, 30, 100, None),
         (200, 130, 300, [0, 100, 100, 101, 133, 133, 190, 196, 197]), (90, 600, 2100, [3, 40, 90])]


@pytest.mark.parametrize("case", range(len(SMALL)))
def test_small_products(nv, case):
    M, N, K, off = SMALL[case]
    print(f"small {case}", flush=True)
    a, b = copy_of(nv, (M,), K, 41), copy_of(nv, (N,) if off is None else (len(off) - 1, N), K, 42)
    av, bv = values(a), values(b)
    for dt, name in DTYPES:
        if off is None:
            check(nv.mxfp4_gemm(a, b, out_dtype=dt), *product(av, bv), f"small {name}")
            continue
        c = nv.mxfp4_gemm_grouped(a, b, torch.tensor(off, dtype=torch.int32, device=dev()), out_dtype=dt)
        inside = torch.zeros(M, dtype=torch.bool, device=dev())
        for g, (i, j) in enumerate(ref.spans(off, M)):
            inside[i:j] = True
            if j > i:
                check(c[i:j], *product(av[i:j], bv[g]), f"small {name}")
        assert (c[~inside] == 0).all()


@pytest.mark.parametrize("M,N,K", [(17, 100, 300), (32, 1024, 1000), (40, 1000, 96), (64, 1024, 1030), (100, 2100, 130),
                                   (250, 1000, 513), (1000, 500, 64), (33, 4500, 520), (2, 9000, 1000), (5, 9000, 3000)])
def test_small_linear(nv, M, N, K):
    """The quantization inside the product at every tile of it, and as its own kernel beyond."""
    print(f"small linear {M}x{N}x{K}", flush=True)
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(M, K + 3, device=dev()).to(dtype)[:, 1:1 + K]
        w = copy_of(nv, (N,), K, 45)
        for rule in (ref.FLOOR, ref.CEIL):
            q = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(scale_rule=rule))[0]
            want, absdot = product(values(q), values(w))
            for dt, name in DTYPES:
                check(nv.mxfp4_linear(x, w, scale_rule=rule, out_dtype=dt), want, absdot, f"linear {name}")


def test_nan_blocks_stay_in_their_rows_and_columns(nv):
    """A NaN block makes its row of C, and only that, NaN; whatever tile the product takes."""
    for M, N, K in [(16, 40, 700), (24, 4000, 300), (64, 300, 2080), (700, 600, 300), (2304, 2560, 320)]:
        a, b = copy_of(nv, (M,), K, 43), copy_of(nv, (N,), K, 44)
        a.scales[M - 3, 1], b.scales[5, -(-K // 32) - 1] = 255, 255
        want, absdot = product(torch.nan_to_num(values(a)), torch.nan_to_num(values(b)))
        c = nv.mxfp4_gemm(a, b)
        nan = torch.zeros(M, N, dtype=torch.bool, device=dev())
        nan[M - 3], nan[:, 5] = True, True
        assert torch.equal(torch.isnan(c), nan)
        keep = ~nan
        check(c[keep], want[keep], absdot[keep], "beside NaN")


def test_large_tiles_with_one_row_and_short_k(nv):
    """Tiles of one row or column, K of less than a stage, groups of no and of one row of K."""
    for M, N, K in [(4097, 4096, 30), (4096, 4097, 130), (4097, 4097, 1)]:
        a, b = copy_of(nv, (M,), K, 31), copy_of(nv, (N,), K, 32)
        check(nv.mxfp4_gemm(a, b), *product(values(a), values(b)), f"dense {M}x{N}x{K}")
    M, N, K, off = 8195, 2049, 50, [0, 1, 2, 2, 8194]
    a, b = copy_of(nv, (M,), K, 33), copy_of(nv, (4, N), K, 34)
    c = nv.mxfp4_gemm_grouped(a, b, torch.tensor(off, dtype=torch.int32, device=dev()))
    av, bv = values(a), values(b)
    for g, (i, j) in enumerate(ref.spans(off, M)):
        if j > i:
            check(c[i:j], *product(av[i:j], bv[g]), "grouped")
    assert (c[8194:] == 0).all()
    off = torch.tensor([0, 1, 1, 5], dtype=torch.int32, device=dev())
    p = nv.mxfp4_quant_params(False, True)
    x, y = torch.randn(5, 2048, device=dev()), torch.randn(5, 2049, device=dev())
    xc, yc = (nv.mxfp4_quantize(t, p, offsets=off)[1] for t in (x, y))
    c = nv.mxfp4_gemm_grouped_wgrad(xc, yc, off)
    xv, yv = values(xc), values(yc)
    for g, (i, j) in enumerate([(0, 128), (128, 128), (128, 256)]):
        check(c[g], *product(xv[:, i:j], yv[:, i:j]), "wgrad")


def test_gradients_against_formula(nv):
    """dX and dW of Y = X W^T from row and column copies, in 64 bits from the copies' values."""
    for T, N, K in [(100, 60, 70), (513, 300, 257), (1100, 520, 640)]:
        x, w, dy = torch.randn(T, K, device=dev()), torch.randn(N, K, device=dev()), torch.randn(T, N, device=dev())
        p = nv.mxfp4_quant_params(True, True, ref.CEIL)
        (xr, xc), (wr, wc), (dyr, dyc) = (nv.mxfp4_quantize(t, p) for t in (x, w, dy))
        check(nv.mxfp4_gemm(xr, wr), *product(values(xr), values(wr)), "Y f32")
        check(nv.mxfp4_gemm(dyr, wc), *product(values(dyr), values(wc)), "dX f32")
        check(nv.mxfp4_gemm(dyc, xc), *product(values(dyc), values(xc)), "dW f32")
        # and they are gradients of the unquantized layer up to the quantization's error: E2M1
        # keeps each value within 1/4 of itself or 1/12 of its block's maximum, on average far less
        for got, exact in ((nv.mxfp4_gemm(dyr, wc), dy.double() @ w.double()),
                           (nv.mxfp4_gemm(dyc, xc), dy.double().t().contiguous() @ x.double())):
            assert ((got - exact).norm() / exact.norm()).item() < 0.25


def test_gradients_against_differences(nv):
    """With operands whose quantization changes nothing (values on the grid of their block, each
    block's maximum fixed), L = <dY, Y(X, W)> is bilinear and central differences with grid steps
    are exact: every sum is of small integers, below 2^24."""
    r = np.random.RandomState(0)
    T, N, K = 40, 36, 70

    def on_grid(n, k):
        v = r.choice([-3.0, -2, -1, 0, 1, 2, 3], (n, k))
        v[:, ::16], v[::16] = 4.0, 4.0            # every row block and column block has amax 4
        return torch.tensor(v, dtype=torch.float32, device=dev())

    x, w, dy = on_grid(T, K), on_grid(N, K), on_grid(T, N)
    p = nv.mxfp4_quant_params(True, True)
    (xr, xc), (wr, wc), (dyr, dyc) = (nv.mxfp4_quantize(t, p) for t in (x, w, dy))
    dx, dw = nv.mxfp4_gemm(dyr, wc), nv.mxfp4_gemm(dyc, xc)

    def loss(x, w):
        return (nv.mxfp4_gemm(nv.mxfp4_quantize(x, p)[0], nv.mxfp4_quantize(w, p)[0]).double() * dy.double()).sum().item()

    for t, grad, f in ((x, dx, lambda v: loss(v, w)), (w, dw, lambda v: loss(x, v))):
        for i, j in [(1, 1), (5, 33), (17, 69), (35, 47)]:
            hi, lo = t.clone(), t.clone()
            hi[i, j], lo[i, j] = 2.0, 0.0
            assert (f(hi) - f(lo)) / 2 == grad[i, j].item()


def test_linear_on_another_stream_and_in_a_graph(nv):
    x = torch.randn(33, 640, device=dev()).bfloat16()
    w = copy_of(nv, (700,), 640, 9)
    off = torch.tensor([0, 10, 33], dtype=torch.int32, device=dev())
    w2 = copy_of(nv, (2, 300), 640, 10)
    need = max(nv.mxfp4_linear_workspace_bytes(33, 700, 640), nv.mxfp4_linear_workspace_bytes(33, 300, 640, 2))
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    big, bigw = copy_of(nv, (600,), 640, 11), copy_of(nv, (512,), 640, 12)
    eager = [nv.mxfp4_linear(x, w), nv.mxfp4_linear(x, w2, offsets=off), nv.mxfp4_gemm(big, bigw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = [nv.mxfp4_linear(x, w), nv.mxfp4_linear(x, w2, offsets=off), nv.mxfp4_gemm(big, bigw)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    outs = [torch.empty_like(t) for t in eager]

    def chain():
        nv.mxfp4_linear(x, w, out=outs[0], workspace=ws)
        nv.mxfp4_linear(x, w2, offsets=off, out=outs[1], workspace=ws)
        nv.mxfp4_gemm(big, bigw, out=outs[2])

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for i in range(3):
        for o in outs:
            o.fill_(float(i))
        off.copy_(torch.tensor([0, 10 + i, 33], dtype=torch.int32))     # offsets are read on the device
        want = nv.mxfp4_linear(x, w2, offsets=off)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager[0]) and torch.equal(outs[1], want) and torch.equal(outs[2], eager[2])


def test_empty(nv):
    d = dev()
    e = lambda n, k: nv.MXTensor.empty(n, k, d)
    assert nv.mxfp4_gemm(e(0, 5), e(7, 5)).shape == (0, 7)
    assert nv.mxfp4_gemm(e(7, 5), e(0, 5)).shape == (7, 0)
    assert (nv.mxfp4_gemm(e(3, 0), e(4, 0), out=torch.ones(3, 4, device=d)) == 0).all()
    assert (nv.mxfp4_linear(torch.empty(3, 0, device=d), e(4, 0), out=torch.ones(3, 4, device=d)) == 0).all()
    off = torch.tensor([0, 0, 0], dtype=torch.int32, device=d)
    x = torch.empty(0, 40, device=d)
    assert nv.mxfp4_linear(x, e((2, 9), 40), offsets=off).shape == (0, 9)
    col = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(False, True), offsets=off)[1]
    c = nv.mxfp4_gemm_grouped_wgrad(col, col, off, out=torch.ones(2, 40, 40, device=d))
    assert (c == 0).all()


def test_no_k(nv):
    """Products over K = 0 are zeros at every size."""
    d = dev()
    e = lambda n: nv.MXTensor.empty(n, 0, d)
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device=d)
    for M, N in ((1, 1), (16, 300), (40, 700), (600, 700), (4096, 4100)):
        for dt, _ in DTYPES:
            assert (nv.mxfp4_gemm(e(M), e(N), out=torch.ones(M, N, device=d, dtype=dt)) == 0).all()
            assert (nv.mxfp4_gemm_grouped(e(M), e((2, N)), off, out=torch.ones(M, N, device=d, dtype=dt)) == 0).all()


def test_refusals(nv):
    d = dev()
    e = lambda n, k, g=0: nv.MXTensor.empty(n, k, d, g)
    off = torch.tensor([0, 8], dtype=torch.int32, device=d)
    x = torch.zeros(8, 64, device=d)
    bad = [lambda: nv.mxfp4_gemm(e(8, 64), e(8, 65)), lambda: nv.mxfp4_gemm(e(8, 64), e((1, 8), 64)),
           lambda: nv.mxfp4_gemm(e(8, 64), e(8, 64, 2)), lambda: nv.mxfp4_gemm(e(8, 64), e(8, 64), out_dtype=torch.half),
           lambda: nv.mxfp4_gemm(e(8, 64), e(8, 64), out=torch.empty(8, 9, device=d)),
           lambda: nv.mxfp4_gemm(e(8, 64), e(8, 64), out=torch.empty(8, 8, device=d).t()[:, ::2]),
           lambda: nv.mxfp4_gemm_grouped(e(8, 64), e((2, 8), 64), off), lambda: nv.mxfp4_gemm_grouped(e(8, 64), e(8, 64), off),
           lambda: nv.mxfp4_gemm_grouped(e(8, 64), e((1, 8), 64), None),
           lambda: nv.mxfp4_gemm_grouped_wgrad(e(8, 64), e(8, 64), off),
           lambda: nv.mxfp4_gemm_grouped_wgrad(e(8, 64, 1), e(8, 63, 1), off),
           lambda: nv.mxfp4_linear(x, e(8, 63)), lambda: nv.mxfp4_linear(x, e((1, 8), 64)),
           lambda: nv.mxfp4_linear(x, e((2, 8), 64), offsets=off), lambda: nv.mxfp4_linear(x.half(), e(8, 64)),
           lambda: nv.mxfp4_linear(x, e(8, 64), scale_rule=2),
           lambda: nv.mxfp4_linear(x.t(), e(8, 8)), lambda: nv.mxfp4_linear(x.repeat(2200, 1), e(8, 64), workspace=torch.empty(1, dtype=torch.uint8, device=d)),
           lambda: nv.mxfp4_gemm(nv.MXTensor(e(8, 64).codes[:, ::2], e(8, 64).scales, 64), e(8, 64)),
           lambda: nv.mxfp4_gemm(nv.MXTensor(e(8, 64).codes.cpu(), e(8, 64).scales, 64), e(8, 64))]
    for i, f in enumerate(bad):
        with pytest.raises(nv.Nvfp4Error):
            f()
            print("not refused:", i)
