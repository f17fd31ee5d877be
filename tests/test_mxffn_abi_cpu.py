"""C ABI of the gated feed-forward block and the checkpoints, without a GPU: exports, the argument
errors that are returned before anything is enqueued, and libraries that lack these functions."""
import ctypes
import os
import re
import subprocess

import pytest

from test_mxfp4_abi_cpu import FAKE, ROOT, nv, nv_c  # noqa: F401  (nv: fixture)

HEADER = os.path.join(ROOT, "include", "mxffn.h")
VP = ctypes.c_void_p


def test_header_exports_and_version(nv):  # noqa: F811
    from nvfp4_block_scaled_quantize_amd import mxffn
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mxf(?:p[48]|fn)_[a-z0-9_]*)\s*\([^;{]*\)\s*;", text)))
    assert names == sorted(mxffn.MXFFN_EXPORTED)
    lib = ctypes.CDLL(nv.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)
    assert nv.load_library().mxffn_abi_version() == mxffn.MXFFN_ABI_VERSION


def test_checkpoint_argument_errors(nv):  # noqa: F811
    lib, q = nv.load_library(), nv_c(FAKE, FAKE + 0x10000)

    def quantize(x=FAKE + 0x20000, dtype=1, batch=1, rows=8, cols=8, ld=8, q=q):
        return lib.mxfp8_quantize(x, dtype, batch, rows, cols, ld, 64, q, None)

    def decode(q=q, n=8, k=8, dtype=0, out=FAKE + 0x20000, ld=8):
        return lib.mxfp8_dequantize(q, n, k, dtype, out, ld, None)

    assert quantize(x=None) == -1 and quantize(q=None) == -1 and quantize(q=nv_c(0, FAKE)) == -1
    assert quantize(rows=-1) == -2 and quantize(cols=-1) == -2 and quantize(batch=-1) == -2 and quantize(ld=7) == -2
    assert quantize(rows=1 << 33, cols=1 << 13, ld=1 << 13) == -2 and quantize(rows=(1 << 34) + 1) == -2
    assert quantize(dtype=2) == -4 and quantize(x=FAKE + 1) == -3 and quantize(x=FAKE + 2, dtype=0) == -3
    assert quantize(q=nv_c(FAKE + 8, FAKE)) == -3 and quantize(q=nv_c(FAKE, FAKE + 2)) == -3
    assert quantize(rows=0, x=None, q=nv_c(0, 0)) == 0 and quantize(batch=0) == 0
    assert decode(q=None) == -1 and decode(out=None) == -1 and decode(q=nv_c(FAKE, 0)) == -1
    assert decode(n=-1) == -2 and decode(k=-1) == -2 and decode(ld=7) == -2 and decode(n=1 << 33, k=1 << 13, ld=1 << 13) == -2
    assert decode(dtype=3) == -4 and decode(out=FAKE + 2) == -3 and decode(out=FAKE + 1, dtype=1) == -3
    assert decode(n=0, q=nv_c(0, 0), out=None) == 0 and decode(k=0, out=None) == 0
    P = nv.mxfp4_quant_params
    off = VP(FAKE + 0x70000)
    row, col = nv_c(FAKE + 0x20000, FAKE + 0x30000), nv_c(FAKE + 0x40000, FAKE + 0x50000)

    def copies(q=q, batch=1, rows=8, cols=8, offsets=None, groups=0, p=P(True, True), row=row, col=col):
        return lib.mxfp8_to_mxfp4(q, batch, rows, cols, offsets, groups, p, row, col, None)

    assert copies(q=None) == -1 and copies(p=None) == -1 and copies(row=None) == -1 and copies(col=None) == -1
    assert copies(batch=-1) == -2 and copies(rows=-1) == -2 and copies(cols=-1) == -2 and copies(groups=-1) == -2
    assert copies(p=P(False, False)) == -5 and copies(p=P(True, False, 3)) == -5 and copies(p=P(True, True, 0, 2)) == -5
    assert copies(offsets=off) == -5 and copies(groups=2) == -1 and copies(groups=2, offsets=off, batch=2) == -5
    assert copies(q=nv_c(FAKE + 4, FAKE)) == -3 and copies(col=nv_c(FAKE, FAKE + 1)) == -3
    assert copies(rows=1 << 34, cols=1 << 33) == -2 and copies(rows=0, q=nv_c(0, 0)) == 0


def test_gated_argument_errors(nv):  # noqa: F811
    lib = nv.load_library()
    a, w, q, k = (nv_c(FAKE + i * 0x20000, FAKE + i * 0x20000 + 0x10000) for i in range(4))
    out, off = VP(FAKE + 0x90000), VP(FAKE + 0xA0000)

    def gated(a=a, w=w, o=None, n=0, M=8, N=8, K=8, act=0, h=out, dt=1, ld=8, rule=0, copy=q, kept=k):
        return lib.mxfp4_gated(a, w, o, n, M, N, K, act, h, dt, ld, rule, copy, kept, None)

    assert gated(a=None) == -1 and gated(w=None) == -1 and gated(h=None, copy=None, kept=None) == -1
    assert gated(copy=nv_c(0, FAKE)) == -1 and gated(kept=nv_c(FAKE, 0)) == -1 and gated(n=2) == -1
    assert gated(M=-1) == -2 and gated(N=-1) == -2 and gated(K=-1) == -2 and gated(ld=7) == -2 and gated(K=(1 << 23) + 1) == -2
    assert gated(N=1 << 34) == -2 and gated(M=1 << 33, N=1 << 10, ld=1 << 10) == -2 and gated(o=off, n=-1) == -2
    assert gated(o=off, n=2, M=1 << 31) == -2
    assert gated(dt=2) == -4 and gated(act=2) == -5 and gated(act=-1) == -5 and gated(rule=2) == -5 and gated(o=off) == -5
    assert gated(h=VP(FAKE + 1)) == -3 and gated(h=VP(FAKE + 2), dt=0) == -3 and gated(copy=nv_c(FAKE + 8, FAKE)) == -3
    assert gated(kept=nv_c(FAKE, FAKE + 2)) == -3 and gated(o=VP(FAKE + 2), n=2) == -3 and gated(a=nv_c(FAKE + 4, FAKE)) == -3
    assert gated(M=0, a=nv_c(0, 0), h=None, copy=None, kept=None) == 0 and gated(N=0, w=nv_c(0, 0)) == 0

    def backward(dy=a, w=w, o=None, n=0, M=8, N=8, K=8, act=0, kept=k, g=out, dt=1, ld=16, h=VP(FAKE + 0xB0000), ldh=8):
        return lib.mxfp4_gated_backward(dy, w, o, n, M, N, K, act, kept, g, dt, ld, h, ldh, None)

    assert backward(dy=None) == -1 and backward(w=None) == -1 and backward(kept=None) == -1 and backward(g=None) == -1
    assert backward(n=2) == -1 and backward(kept=nv_c(0, 0)) == -1
    assert backward(M=-1) == -2 and backward(N=-1) == -2 and backward(K=-1) == -2 and backward(ld=15) == -2 and backward(ldh=7) == -2
    assert backward(dt=2) == -4 and backward(act=2) == -5 and backward(o=off) == -5
    assert backward(g=VP(FAKE + 1)) == -3 and backward(h=VP(FAKE + 1)) == -3 and backward(kept=nv_c(FAKE + 1, FAKE)) == -3
    assert backward(M=0, g=None) == 0 and backward(N=0) == 0

    def from_dh(dh=VP(FAKE), ddt=1, ldd=8, M=8, N=8, act=0, kept=k, g=out, dt=1, ld=16, h=VP(FAKE + 0xB0000), ldh=8):
        return lib.mxfp8_gated_backward(dh, ddt, ldd, M, N, act, kept, g, dt, ld, h, ldh, None)

    assert from_dh(dh=None) == -1 and from_dh(kept=None) == -1 and from_dh(g=None) == -1
    assert from_dh(M=-1) == -2 and from_dh(N=-1) == -2 and from_dh(ldd=7) == -2 and from_dh(ld=15) == -2 and from_dh(ldh=7) == -2
    assert from_dh(M=1 << 34, N=1 << 20, ldd=1 << 20, ld=1 << 21, ldh=1 << 20) == -2
    assert from_dh(ddt=2) == -4 and from_dh(dt=2) == -4 and from_dh(act=2) == -5
    assert from_dh(dh=VP(FAKE + 1)) == -3 and from_dh(g=VP(FAKE + 1)) == -3 and from_dh(h=VP(FAKE + 1)) == -3
    assert from_dh(M=0, dh=None, g=None) == 0 and from_dh(h=None, ldh=0, M=0) == 0


def test_gated_linear_argument_errors(nv):  # noqa: F811
    lib, w = nv.load_library(), nv_c(FAKE, FAKE + 0x10000)
    need = lib.mxfp4_gated_linear_workspace_bytes(17000, 8, 8, 0)

    def linear(x=VP(FAKE), dt=1, M=17000, K=8, ld=8, rule=0, w=w, N=8, o=None, n=0, act=0, h=VP(FAKE + 0x40000), hdt=1, ldh=8,
               ws=FAKE + 0x60000, size=1 << 21):
        return lib.mxfp4_gated_linear(x, dt, M, K, ld, rule, w, N, o, n, act, h, hdt, ldh, ws, size, None)

    assert need > 0 and linear(size=need - 1) == -6 and linear(ws=None) == -6 and linear(ws=FAKE + 0x60001) == -3
    for m in (17000, 1):
        assert linear(M=m, x=None) == -1 and linear(M=m, w=None) == -1 and linear(M=m, h=None) == -1
        assert linear(M=m, ld=7) == -2 and linear(M=m, ldh=7) == -2 and linear(M=m, K=-1) == -2 and linear(M=m, N=-1) == -2
        assert linear(M=m, dt=2) == -4 and linear(M=m, hdt=2) == -4
        assert linear(M=m, rule=2) == -5 and linear(M=m, act=2) == -5 and linear(M=m, o=VP(FAKE)) == -5
        assert linear(M=m, x=VP(FAKE + 1)) == -3 and linear(M=m, h=VP(FAKE + 1)) == -3 and linear(M=m, n=2) == -1
    assert linear(M=-1) == -2 and linear(M=0, x=None, h=None) == 0
    for M, N, K in ((1 << 35, 8, 8), (8, 1 << 34, 8), (8, 8, 1 << 24), (-1, 8, 8)):
        assert lib.mxfp4_gated_linear_workspace_bytes(M, N, K, 0) == 0


@pytest.mark.parametrize("kind", ["without", "another version", "with"])
def test_library_that_lacks_them(kind, tmp_path, monkeypatch):
    """The other calls' library is loaded whether or not it has these functions; only they refuse it."""
    import nvfp4_block_scaled_quantize_amd as nv
    from nvfp4_block_scaled_quantize_amd import mxffn, mxfp4
    values = {name: 0 for name in nv.EXPORTED + mxfp4.MXFP4_EXPORTED}
    values["nvfp4_abi_version"], values["mxfp4_abi_version"] = nv.ABI_VERSION, mxfp4.MXFP4_ABI_VERSION
    if kind != "without":
        values |= {name: 0 for name in mxffn.MXFFN_EXPORTED}
        values["mxffn_abi_version"] = mxffn.MXFFN_ABI_VERSION + (kind != "with")
    (tmp_path / "stub.c").write_text("".join(f"long {n}(void) {{ return {v}; }}\n" for n, v in values.items()))
    subprocess.check_call(["gcc", "-shared", "-fPIC", str(tmp_path / "stub.c"), "-o", str(tmp_path / "stub.so")])
    monkeypatch.setattr(nv, "LIB_PATH", str(tmp_path / "stub.so"))
    monkeypatch.setattr(nv, "_lib", None)
    for module in (mxfp4, mxffn):
        monkeypatch.setattr(module, "_bound", None)
        monkeypatch.setattr(module, "_unusable", None)
    if kind == "with":
        assert nv.mxfp4_gated_linear_workspace_bytes(1, 32, 32) == 0
    else:
        for _ in range(2):
            with pytest.raises(nv.Nvfp4Error, match="rebuild"):
                nv.mxfp4_gated_linear_workspace_bytes(1, 32, 32)
    assert nv.mxfp4_linear_workspace_bytes(1, 32, 32) == 0 and nv.load_library().nvfp4_abi_version() == nv.ABI_VERSION


@pytest.mark.parametrize("source", ["mx_ffn_forward128.hip", "mx_ffn_forward256.hip", "mx_ffn_backward128.hip"])
def test_nothing_else_writes_m0(source):
    """As of the plain products' kernels: several direct loads share what one instruction set M0 to."""
    import test_direct_load_m0_cpu
    test_direct_load_m0_cpu.test_nothing_else_writes_m0(source)
