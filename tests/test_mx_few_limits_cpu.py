"""Sizes of few rows whose workgroups in the kernel for few rows do not fit a launch: the calls take the tiled kernels,
whose do, instead of refusing them.  Without a GPU such a call ends where the kernel would be launched."""
import ctypes

import pytest
import torch

from test_mxfp4_abi_cpu import FAKE, nv, nv_c  # noqa: F401  (nv: fixture)

VP = ctypes.c_void_p
HIP = -7
# (M, N, K, groups): 2^24 workgroups of 256 threads or more
SIZES = [(1, 1 << 28, 128, 0), (2, (1 << 28) + 5, 40, 0), (8192, 65536, 128, 8192), (9000, 1 << 17, 100, 4096)]


@pytest.mark.parametrize("M,N,K,groups", SIZES)
def test_workspaces_of_the_layers(nv, M, N, K, groups):  # noqa: F811
    """They are quantized by a kernel of their own, into a workspace."""
    lib = nv.load_library()
    for f in (lib.mxfp4_linear_workspace_bytes, lib.mxfp4_gated_linear_workspace_bytes):
        assert f(M, N, K, groups) >= M * 17 * 4
        assert f(M, 1000, K, 0) == 0 or M > 2     # where the few rows' kernel fits, it quantizes them


@pytest.mark.parametrize("M,N,K,groups", SIZES + [(16, 1 << 28, 128, 0)])
def test_calls(nv, M, N, K, groups):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real: without a GPU alone")
    lib, off = nv.load_library(), VP(FAKE) if groups else None
    a, w, kept, out = nv_c(FAKE, FAKE), nv_c(FAKE, FAKE), nv_c(FAKE, FAKE), VP(FAKE)
    if groups:
        assert lib.mxfp4_gemm_grouped(a, w, off, groups, M, N, K, out, 1, N, None) == HIP
    else:
        assert lib.mxfp4_gemm(a, w, M, N, K, out, 1, N, None) == HIP
    assert lib.mxfp4_gated(a, w, off, groups, M, N, K, 0, out, 1, N, 0, None, None, None) == HIP
    assert lib.mxfp4_gated_backward(a, w, off, groups, M, N, K, 0, kept, out, 1, 2 * N, None, 0, None) == HIP
