"""Extents whose grids do not fit a launch are refused with the shape status before anything is
enqueued.  No call here reaches a kernel: the pointers are never dereferenced."""
import ctypes
import os

import pytest

FAKE = 0x7F0000000000
OK, SHAPE = 0, -2


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not os.path.exists(nv.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build_hip()
    nv.load_library()
    return nv


def copy():
    from nvfp4_block_scaled_quantize_amd.mxfp4 import MXTensorC
    return MXTensorC(FAKE, FAKE + 0x1000)


# (batch, rows, cols, rowwise, colwise, groups): 2^24 workgroups of 256 threads or more
QUANTIZE = [(1, 1 << 30, 1, 1, 0, 0), (1 << 30, 1, 1, 1, 0, 0), (1, 1 << 25, 1 << 13, 1, 0, 0), (1, 1, 1 << 40, 1, 0, 0),
            (1 << 24, 1, 1, 0, 1, 0), (1, 1 << 31, 1, 1, 1, 0), (1, 1, 1 << 31, 0, 1, 0), (1, 1 << 20, 1 << 20, 1, 1, 0),
            (1, (1 << 31) - 70000, 256, 0, 1, 7), (1 << 40, 1 << 10, 1 << 10, 1, 1, 0), (1 << 20, 1 << 30, 1 << 30, 1, 1, 0),
            (1 << 62, 4, 8, 1, 0, 0), ((1 << 63) - 1, 1, 1, 0, 1, 0), (1, (1 << 63) - 1, 1, 1, 1, 0), (1, 1, (1 << 63) - 1, 1, 1, 0)]


@pytest.mark.parametrize("case", QUANTIZE)
def test_quantize(nv, case):
    batch, rows, cols, row, col, groups = case
    p = nv.mxfp4_quant_params(row, col)
    off = ctypes.c_void_p(FAKE + 0x70000) if groups else None
    for dtype in (0, 1):
        assert nv.load_library().mxfp4_quantize(FAKE, dtype, batch, rows, cols, cols, rows * cols % (1 << 62), off, groups, p,
                                                copy(), copy(), None) == SHAPE


# (n, k, groups)
DEQUANTIZE = [(1 << 30, 1, 0), (1 << 25, 1 << 13, 0), (1, 1 << 40, 0), (1 << 28, 1 << 13, 3), (1 << 20, (1 << 31) - 70000, 5),
              (1 << 62, 128, 0), ((1 << 63) - 1, 1, 0), (1, (1 << 63) - 1, 0), ((1 << 63) - 1, 1, 1)]


@pytest.mark.parametrize("n,k,groups", DEQUANTIZE)
def test_dequantize(nv, n, k, groups):
    off = ctypes.c_void_p(FAKE + 0x70000) if groups else None
    for dtype in (0, 1):
        assert nv.load_library().mxfp4_dequantize(copy(), n, k, off, groups, dtype, FAKE + 0x100000, k, None) == SHAPE


# (M, N, K, groups)
PRODUCTS = [(1 << 31, 1 << 10, 32, 0), (1 << 24, 1 << 24, 32, 0), (1 << 40, 1, 32, 0), (1, 1 << 40, 32, 0),
            (1 << 30, 1 << 12, 32, 4), ((1 << 63) - 1, 1, 32, 0), (1, (1 << 63) - 1, 32, 0), (1, (1 << 63) - 1, 32, 3)]


@pytest.mark.parametrize("M,N,K,groups", PRODUCTS)
def test_products(nv, M, N, K, groups):
    lib = nv.load_library()
    off = ctypes.c_void_p(FAKE + 0x70000)
    for dtype in (0, 1):
        if groups:
            assert lib.mxfp4_gemm_grouped(copy(), copy(), off, groups, M, N, K, FAKE, dtype, N, None) == SHAPE
        else:
            assert lib.mxfp4_gemm(copy(), copy(), M, N, K, FAKE, dtype, N, None) == SHAPE
        assert lib.mxfp4_gemm_grouped_wgrad(copy(), copy(), off, 3, M, N, 64, FAKE, dtype, N, None) == SHAPE


@pytest.mark.parametrize("M,N,K,groups", PRODUCTS)
def test_linear(nv, M, N, K, groups):
    lib = nv.load_library()
    off = ctypes.c_void_p(FAKE + 0x70000) if groups else None
    for dtype in (0, 1):
        assert lib.mxfp4_linear(FAKE, 1, M, K, K, 0, copy(), N, off, groups, FAKE, dtype, N, ctypes.c_void_p(FAKE),
                                (1 << 64) - 1, None) == SHAPE
        assert lib.mxfp4_linear_workspace_bytes(M, N, K, groups) == 0


def test_sizes_of_the_workspace(nv):
    """0 for sizes that mxfp4_linear refuses, whatever their product wraps to."""
    f = nv.load_library().mxfp4_linear_workspace_bytes
    assert f(17000, 1 << 30, 8, 0) == 0 and f(17000, 8, (1 << 23) + 1, 0) == 0 and f(-1, 8, 8, 0) == 0
    assert f(17000, 8, 8, 0) > 0
