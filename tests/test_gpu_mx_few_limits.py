"""Few rows through more columns than the kernel for few rows has workgroups for (2^28): the tiled kernels take them."""
import pytest
import torch

import mxffn_reference as ref
from gpu_util import dev
from test_gpu_mxffn import check_forward, nv  # noqa: F401  (nv: fixture)
from test_gpu_mxfp4_gemm import check, copy_of, product, values

pytestmark = pytest.mark.gpu


def test_more_columns_than_workgroups(nv):  # noqa: F811
    M, N, K = 2, (1 << 28) + 40, 128
    need = 2 * N * 68 + 3 * M * N * 2
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip("not enough memory")
    codes = torch.empty(2 * N, 64, dtype=torch.uint8, device=dev())
    for part in codes.split(1 << 24):
        part.random_(0, 256)
    w = nv.MXTensor(codes, torch.empty(2 * N, 4, dtype=torch.uint8, device=dev()).random_(118, 121), K)
    x = torch.randn(M, K, device=dev()).bfloat16()
    a = nv.mxfp4_quantize(x, nv.mxfp4_quant_params())[0]
    some = torch.cat([torch.arange(0, 40), torch.randint(0, N, (200,)), torch.arange(N - 40, N)]).to(dev())
    part = lambda rows: nv.MXTensor(w.codes[rows], w.scales[rows], K)
    half = nv.MXTensor(w.codes[:N], w.scales[:N], K)
    for c in (nv.mxfp4_gemm(a, half, out_dtype=torch.bfloat16), nv.mxfp4_linear(x, half)):
        check(c[:, some], *product(values(a), values(part(some))), "product")
    for h in (nv.mxfp4_gated(a, w)[0], nv.mxfp4_gated_linear(x, w)):
        check_forward(nv, a, part(torch.cat([some, some + N])), some.numel(), (h[:, some], None, None), ref.SILU, 0, "gated")


def test_groups_of_a_row_each(nv):  # noqa: F811
    """8192 experts of 65536 rows: 2^24 workgroups of 32 columns and one row."""
    M, N, K = 8192, 65536, 128
    if torch.cuda.mem_get_info()[0] < M * N * 68 + 3 * M * N * 2 + (8 << 30):
        pytest.skip("not enough memory")
    codes, scales = torch.empty(M, N, 64, dtype=torch.uint8, device=dev()), torch.full((M, N, 4), 120, dtype=torch.uint8, device=dev())
    for part in codes.split(256):
        part.random_(0, 256)
    w, a = nv.MXTensor(codes, scales, K), copy_of(nv, (M,), K, 3, spread=1)
    offsets = torch.arange(M + 1, dtype=torch.int32, device=dev())
    c = nv.mxfp4_gemm_grouped(a, w, offsets, out_dtype=torch.bfloat16)
    for e in (0, 1, 4097, M - 1):
        one = nv.MXTensor(a.codes[e:e + 1].contiguous(), a.scales[e:e + 1].contiguous(), K)
        check(c[e:e + 1], *product(values(one), values(nv.MXTensor(w.codes[e], w.scales[e], K))), f"expert {e}")
