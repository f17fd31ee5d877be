"""MXFP4 C ABI checks that need no GPU: exports, sizes, and the argument errors that are
returned before anything is enqueued; and pins of the tests' own reference."""
import ctypes
import os
import re

import numpy as np
import pytest

import mxfp4_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxfp4.h")
FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not os.path.exists(nv.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build_hip()
    nv.load_library()
    return nv


def test_header_exports_and_version(nv):
    from nvfp4_block_scaled_quantize_amd import mxfp4
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mxfp4_[a-z0-9_]*)\s*\([^;{]*\)\s*;", text)))
    assert names == sorted(mxfp4.MXFP4_EXPORTED)
    lib = ctypes.CDLL(nv.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)
    assert nv.load_library().mxfp4_abi_version() == mxfp4.MXFP4_ABI_VERSION


def test_extents(nv):
    from nvfp4_block_scaled_quantize_amd import mxfp4
    lib = nv.load_library()
    r = np.random.RandomState(0)
    for k in [0, 1, 127, 128, 129, 5000]:
        assert lib.mxfp4_padded_k(k) == mxfp4.padded_k(k) == ref.pad128(k)
    for _ in range(300):
        rows, groups = int(r.randint(0, 3000)), int(r.randint(1, 80))
        kp = lib.mxfp4_grouped_k(rows, groups)
        assert kp == mxfp4.grouped_k(rows, groups) and kp % 128 == 0
        off = np.r_[0, np.sort(r.randint(0, rows + 1, groups - 1)), rows]
        assert ref.grouped_positions(off, rows)[2] <= kp
        # one row per group first, the rest in the last: the most padding there can be
        worst = np.minimum(np.r_[np.arange(groups), rows], rows)
        assert ref.grouped_positions(worst, rows)[2] <= kp



def nv_c(codes, scales):
    from nvfp4_block_scaled_quantize_amd.mxfp4 import MXTensorC
    return MXTensorC(codes, scales)


def test_quantize_argument_errors(nv):
    lib, q = nv.load_library(), nv_c(FAKE, FAKE + 0x10000)
    P = nv.mxfp4_quant_params
    off = ctypes.c_void_p(FAKE + 0x70000)

    def call(x=FAKE + 0x20000, dtype=1, batch=1, rows=8, cols=8, ld=8, offsets=None, groups=0, p=P(True, True),
             row=q, col=q):
        return lib.mxfp4_quantize(x, dtype, batch, rows, cols, ld, 64, offsets, groups, p, row, col, None)

    assert call(p=None) == -1 and call(row=None) == -1 and call(col=None) == -1 and call(x=None) == -1
    assert call(rows=-1) == -2 and call(cols=-1) == -2 and call(batch=-1) == -2 and call(ld=7) == -2
    assert call(groups=-1) == -2 and call(groups=1 << 20, offsets=off) == -2
    assert call(groups=2, offsets=off, rows=1 << 31) == -2
    assert call(dtype=2) == -4
    assert call(p=P(False, False)) == -5 and call(p=P(True, False, 3)) == -5 and call(p=P(True, True, 0, 0, 2)) == -5
    assert call(offsets=off) == -5 and call(groups=2) == -1 and call(groups=2, offsets=off, batch=2) == -5
    assert call(offsets=ctypes.c_void_p(FAKE + 2), groups=2) == -3
    assert call(x=FAKE + 1) == -3 and call(x=FAKE + 2, dtype=0) == -3
    assert call(row=nv_c(FAKE + 8, FAKE)) == -3 and call(col=nv_c(FAKE, FAKE + 2)) == -3
    assert call(rows=0, x=None, row=nv_c(0, 0), col=nv_c(0, 0)) == 0 and call(batch=0) == 0


def test_product_argument_errors(nv):
    lib, a, b = nv.load_library(), nv_c(FAKE, FAKE + 0x10000), nv_c(FAKE + 0x20000, FAKE + 0x30000)
    c, off = ctypes.c_void_p(FAKE + 0x40000), ctypes.c_void_p(FAKE + 0x50000)
    g = lambda a=a, b=b, M=8, N=8, K=8, c=c, dt=0, ldc=8: lib.mxfp4_gemm(a, b, M, N, K, c, dt, ldc, None)
    assert g(a=None) == -1 and g(b=None) == -1 and g(c=None) == -1 and g(a=nv_c(0, FAKE)) == -1
    assert g(M=-1) == -2 and g(N=-1) == -2 and g(K=-1) == -2 and g(ldc=7) == -2 and g(K=(1 << 23) + 1) == -2
    assert g(dt=2) == -4 and g(c=ctypes.c_void_p(FAKE + 2)) == -3 and g(c=ctypes.c_void_p(FAKE + 1), dt=1) == -3
    assert g(a=nv_c(FAKE + 4, FAKE)) == -3 and g(M=0, c=None, a=nv_c(0, 0)) == 0
    r = lambda o=off, n=2, **k: lib.mxfp4_gemm_grouped(a, b, o, n, k.get("M", 8), 8, 8, c, 0, 8, None)
    assert r(o=None) == -1 and r(n=0) == -2 and r(n=-1) == -2 and r(M=1 << 31) == -2 and r(M=0) == 0
    w = lambda o=off, n=2, rows=8, M=8: lib.mxfp4_gemm_grouped_wgrad(a, b, o, n, M, 8, rows, c, 0, 8, None)
    assert w(o=None) == -1 and w(n=0) == -2 and w(rows=-1) == -2 and w(rows=1 << 24) == -2 and w(M=0) == 0
    need = lib.mxfp4_linear_workspace_bytes(17000, 8, 8, 0)
    ln = lambda ws=FAKE + 0x60000, size=1 << 21, rule=0, K=8, ld=8, x=FAKE, N=8, o=None, n=0, dt=1, M=17000: \
        lib.mxfp4_linear(x, dt, M, K, ld, rule, b, N, o, n, c, 0, 8, ws, size, None)
    assert need > 0 and ln(size=need - 1) == -6 and ln(ws=None) == -6
    assert lib.mxfp4_linear_workspace_bytes(1, 8, 8, 0) == 0     # quantized inside the product
    for m in (17000, 1):
        assert ln(M=m, ws=FAKE + 16) == -3 and ln(M=m, rule=2) == -5 and ln(M=m, ld=7) == -2
        assert ln(M=m, K=-1) == -2 and ln(M=m, N=-1) == -2 and ln(M=m, x=None) == -1
        assert ln(M=m, dt=3) == -4 and ln(M=m, n=2) == -1 and ln(M=m, o=off) == -5
        assert ln(M=m, x=FAKE + 1) == -3
    d = lambda **k: lib.mxfp4_dequantize(k.get("q", a), k.get("n", 8), k.get("k", 8), k.get("o"), k.get("g", 0),
                                         k.get("dt", 0), k.get("out", c), k.get("ld", 8), None)
    assert d(q=None) == -1 and d(out=None) == -1 and d(n=-1) == -2 and d(k=-1) == -2 and d(ld=7) == -2
    assert d(dt=5) == -4 and d(out=ctypes.c_void_p(FAKE + 2)) == -3 and d(o=off) == -5 and d(g=1) == -1
    assert d(n=0, out=None) == 0


def test_binding_refuses_cpu_tensors(nv):
    import torch
    with pytest.raises(nv.Nvfp4Error):
        nv.mxfp4_quantize(torch.zeros(4, 32), nv.mxfp4_quant_params())
    q = nv.MXTensor.empty(4, 32, "cpu")
    for f in (lambda: nv.mxfp4_gemm(q, q), lambda: nv.mxfp4_dequantize(q), lambda: nv.mxfp4_linear(torch.zeros(4, 32), q)):
        with pytest.raises(nv.Nvfp4Error):
            f()


def test_reference_philox_matches_the_oracle(oracle):
    r = np.random.RandomState(1)
    ctr = r.randint(0, 2 ** 32, (20, 4), dtype=np.uint64).astype(np.uint32)
    got = ref.philox_words(ctr, 0x0123456789ABCDEF)
    for i in range(20):
        want = oracle.philox4x32_10(ctr[i], np.array([0x89ABCDEF, 0x01234567], np.uint32))
        assert np.array_equal(got[i], np.asarray(want))


def test_reference_rounding_by_hand():
    x = np.zeros((1, 32))
    x[0, :12] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.3, 0, -6, 5.01]
    nib, sc = ref.quantize_rows(x)
    assert sc[0, 0] == 127
    assert (ref.decode(nib, sc)[0, :12] == [6, 4, 4, 2, 2, 1, 1, 0, -0.5, 0, -6, 6]).all()
    assert ref.quantize_rows(np.full((1, 32), 7.0))[1][0, 0] == 127        # saturates
    assert ref.quantize_rows(np.full((1, 32), 7.0), ref.CEIL)[1][0, 0] == 128
    assert ref.quantize_rows(np.full((1, 32), 6.0), ref.CEIL)[1][0, 0] == 127
    assert ref.quantize_rows(np.full((1, 32), np.inf))[1][0, 0] == 255


def test_calls_run_on_their_tensors_device(monkeypatch):
    """A call whose tensors are on another device than the current one switches to it for the call."""
    import contextlib
    from nvfp4_block_scaled_quantize_amd import mxfp4
    entered = []

    @contextlib.contextmanager
    def device(d):
        entered.append(d)
        yield
        entered.append("left")

    monkeypatch.setattr(mxfp4, "_current", lambda: 0)
    monkeypatch.setattr(mxfp4, "_stream", lambda d: 100 + d)
    monkeypatch.setattr(mxfp4.torch.cuda, "device", device)
    seen = []
    f = lambda *a: seen.append((list(entered), a)) or 0
    mxfp4._call(f, 0, 5)
    mxfp4._call(f, 1, 6)
    assert seen == [([], (5, 100)), ([1], (6, 101))] and entered == [1, "left"]


def test_copies_hold_codes_and_scales_in_one_buffer():
    import torch
    import nvfp4_block_scaled_quantize_amd as nv
    for n, k, groups in ((5, 300, 0), ((2, 3), 64, 0), (7, 130, 4), (0, 10, 0), (4, 0, 0), ((0, 3), 5, 0)):
        kp = (k + min(k, groups) * 127) // 128 * 128 if groups else (k + 127) // 128 * 128
        lead = n if isinstance(n, tuple) else (n,)
        t = nv.MXTensor.empty(n, k, "cpu", groups)
        assert t.shape == (*lead, k) and t.codes.shape == (*lead, kp // 2) and t.scales.shape == (*lead, kp // 32)
        t.codes.fill_(1), t.scales.fill_(2)
        assert t.codes.is_contiguous() and t.scales.is_contiguous()
        assert (t.codes == 1).all() and (t.scales == 2).all()          # they do not overlap
        assert t.codes.numel() == 0 or t.scales.data_ptr() == t.codes.data_ptr() + t.codes.numel()
        c = torch.zeros_like(t.codes)
        t.codes = c                                                      # assigned ones are taken as they are
        assert t.codes is c and (t.scales == 2).all() and t.shape == (*lead, k)
    assert "MXTensor" in repr(nv.MXTensor.empty(3, 5, "cpu"))
