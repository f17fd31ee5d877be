"""MXFP4 kernels that only products between the ordinary test sizes take, against 64-bit products: the
quantization inside 32 x 16 tiles, and gradients of groups in more 128 x 128 tiles than compute units."""
import pytest
import torch

import mxfp4_reference as ref
from gpu_util import dev
from test_gpu_mxfp4_gemm import DTYPES, check, copy_of, many_offsets, product, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load_library()
    return nv


@pytest.mark.parametrize("M,N,K", [(64, 1100, 1000), (33, 1500, 130), (50, 2047, 1536), (100, 1000, 700), (200, 570, 31)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear(nv, M, N, K, dtype):
    print(f"linear {M}x{N}x{K} {dtype}", flush=True)
    x = torch.randn(M, K + 3, device=dev()).to(dtype)[:, 1:1 + K]
    w = copy_of(nv, (N,), K, 71)
    for rule in (ref.FLOOR, ref.CEIL):
        q = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(scale_rule=rule))[0]
        want, absdot = product(values(q), values(w))
        for dt, name in DTYPES:
            got = nv.mxfp4_linear(x, w, scale_rule=rule, out_dtype=dt)
            check(got, want, absdot, f"linear {name}")
            assert torch.equal(got, nv.mxfp4_gemm(q, w, out_dtype=dt))


@pytest.mark.parametrize("rows,N,K,G", [(2000, 100, 3000, 30), (3000, 129, 1100, 75), (700, 383, 500, 40)])
def test_wgrad(nv, rows, N, K, G):
    print(f"wgrad {rows} rows {G}x{N}x{K}", flush=True)
    off = many_offsets(rows, G, 72, 30)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    gen = torch.Generator(device=dev()).manual_seed(73)
    p = nv.mxfp4_quant_params(False, True, ref.CEIL)
    dyc, xc = (nv.mxfp4_quantize(torch.randn(rows, n, generator=gen, device=dev()), p, offsets=offsets)[1] for n in (N, K))
    dyv, xv = (nv.mxfp4_dequantize(q, offsets=offsets).double() for q in (dyc, xc))
    for dt, name in DTYPES:
        c = nv.mxfp4_gemm_grouped_wgrad(dyc, xc, offsets, out=torch.full((G, N, K), float("nan"), dtype=dt, device=dev()))
        for g, (i, j) in enumerate(ref.spans(off, rows)):
            if j > i:
                check(c[g], *product(dyv[:, i:j], xv[:, i:j]), f"group {g} {name}")
            else:
                assert (c[g] == 0).all()
