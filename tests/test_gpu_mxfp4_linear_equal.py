"""mxfp4_linear gives what mxfp4_quantize and the product give, bit for bit: whichever kernels it
takes, sums are added in the same order."""
import pytest
import torch

from gpu_util import GEMM_TOL, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load_library()
    return nv


def uneven(*shape):
    """Normal values times powers of two from block to block, so that FP32 sums depend on their order."""
    v = torch.randn(*shape[:-1], -(-shape[-1] // 32), 32, device=dev())
    v *= torch.exp2(torch.randint(-10, 11, (*v.shape[:-1], 1), device=dev()).float())
    return v.flatten(-2)[..., :shape[-1]].contiguous()


DENSE = [(1, 6144, 4096), (1, 70, 30000), (2, 1000, 9000), (7, 16384, 300), (16, 2048, 2048), (33, 700, 512), (64, 1024, 768),
         (100, 1500, 260), (250, 1000, 130), (77, 4999, 2056), (300, 600, 1000)]
# (rows, N, K, ends of the groups): few and many rows a group, at either side of the rules
GROUPED = [(24, 4096, 2048, [2, 2, 7, 11, 24]), (100, 1024, 512, [12, 25, 37, 50, 62, 75, 87, 100]),
           (100, 4096, 512, [0, 0, 60, 61, 61, 100]), (97, 300, 130, [97]), (400, 1536, 256, list(range(16, 401, 16))),
           (200, 65, 600, [10, 100, 100, 150]), (1000, 2048, 96, [5, 200, 999]), (300, 4096, 640, list(range(12, 301, 12))),
           (1100, 520, 64, [100 * i for i in range(12)]), (500, 1999, 333, [0, 33, 65, 65, 130, 300, 301, 480]),
           (333, 3001, 700, [7, 7, 330])]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rule", [0, 1])
def test_dense(nv, dtype, rule):
    for M, N, K in DENSE:
        print(f"dense {M}x{N}x{K} {dtype} {rule}", flush=True)
        x = uneven(M, K).to(dtype)
        w = nv.mxfp4_quantize(uneven(N, K), nv.mxfp4_quant_params())[0]
        q = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(scale_rule=rule))[0]
        for out in (torch.float32, torch.bfloat16):
            assert torch.equal(nv.mxfp4_linear(x, w, scale_rule=rule, out_dtype=out), nv.mxfp4_gemm(q, w, out_dtype=out))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped(nv, case, dtype):
    M, N, K, ends = GROUPED[case]
    print(f"grouped {case} {dtype}", flush=True)
    offsets = torch.tensor([0, *ends], dtype=torch.int32, device=dev())
    x = uneven(M, K).to(dtype)
    w = nv.mxfp4_quantize(uneven(len(ends), N, K), nv.mxfp4_quant_params())[0]
    q = nv.mxfp4_quantize(x, nv.mxfp4_quant_params())[0]
    for out in (torch.float32, torch.bfloat16):
        got = nv.mxfp4_linear(x, w, offsets=offsets, out_dtype=out)
        assert torch.equal(got, nv.mxfp4_gemm_grouped(q, w, offsets, out_dtype=out))
        if out is torch.bfloat16:
            continue
        # |error| <= GEMM_TOL * sum |a b|: products are exact, only the FP32 accumulation rounds
        qv, start = nv.mxfp4_dequantize(q).double(), 0
        wv = nv.mxfp4_dequantize(w).double()
        for e, end in enumerate(ends):
            a, b = qv[start:end], wv[e].t().contiguous()
            assert ((got[start:end] - a @ b).abs() <= GEMM_TOL * (a.abs() @ b.abs())).all()
            start = end
        assert (got[start:] == 0).all()
