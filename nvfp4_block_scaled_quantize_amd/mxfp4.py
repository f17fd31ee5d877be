"""Binding of the MXFP4 operators (C ABI in ``include/mxfp4.h``, built into ``libnvfp4.so``).

MXFP4: E2M1 elements with one E8M0 (power-of-two) scale per 32, the operand format of
gfx950's block-scaled matrix instructions.  As in the package's NVFP4 binding, this module
only marshals arguments; there is no CPU path.

  mxfp4_quantize            rowwise and/or columnwise copies of a bf16/fp32 matrix, or a stack
                            of matrices, or a matrix whose rows are grouped by expert
  mxfp4_dequantize          the values of a copy
  mxfp4_gemm                C = A B^T over two copies
  mxfp4_gemm_grouped        the same with A's rows grouped by expert, one B per expert
  mxfp4_gemm_grouped_wgrad  per expert, C_g = A_g B_g^T over the expert's span of K
  mxfp4_linear              Y = Q(x) W^T in one call, optionally grouped by expert

``offsets`` is a CUDA int32 tensor of n_groups + 1 entries on the operands' device: group g
holds rows offsets[g] .. offsets[g+1].  It stays on the device; no call reads it on the host.
"""
import ctypes
from dataclasses import dataclass

import torch

MXFP4_SCALE_FLOOR, MXFP4_SCALE_CEIL = 0, 1
MXFP4_ABI_VERSION = 1   # MXFP4_ABI_VERSION of include/mxfp4.h this binding matches

MXFP4_EXPORTED = ["mxfp4_padded_k", "mxfp4_grouped_k", "mxfp4_quantize", "mxfp4_dequantize",
                  "mxfp4_gemm", "mxfp4_gemm_grouped", "mxfp4_gemm_grouped_wgrad",
                  "mxfp4_linear_workspace_bytes", "mxfp4_linear", "mxfp4_abi_version"]

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}   # NVFP4_F32, NVFP4_BF16


class MxQuantParams(ctypes.Structure):
    _fields_ = [("rowwise", ctypes.c_int32), ("colwise", ctypes.c_int32),
                ("scale_rule", ctypes.c_int32), ("round_row", ctypes.c_int32),
                ("round_col", ctypes.c_int32), ("seed", ctypes.c_uint64)]


class MXTensorC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


def _error(msg):
    from . import Nvfp4Error
    return Nvfp4Error(msg)


def bind(lib):
    """Declares the MXFP4 functions' types on a loaded libnvfp4.so."""
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    it = ctypes.c_int
    T, Q = ctypes.POINTER(MXTensorC), ctypes.POINTER(MxQuantParams)
    for name, res, args in [
            ("mxfp4_padded_k", i64, [i64]),
            ("mxfp4_grouped_k", i64, [i64, i64]),
            ("mxfp4_quantize", it, [vp, it, i64, i64, i64, i64, i64, vp, i64, Q, T, T, vp]),
            ("mxfp4_dequantize", it, [T, i64, i64, vp, i64, it, vp, i64, vp]),
            ("mxfp4_gemm", it, [T, T, i64, i64, i64, vp, it, i64, vp]),
            ("mxfp4_gemm_grouped", it, [T, T, vp, i64, i64, i64, i64, vp, it, i64, vp]),
            ("mxfp4_gemm_grouped_wgrad", it, [T, T, vp, i64, i64, i64, i64, vp, it, i64, vp]),
            ("mxfp4_linear_workspace_bytes", sz, [i64, i64, i64, i64]),
            ("mxfp4_linear", it, [vp, it, i64, i64, i64, i32, T, i64, vp, i64, vp, it, i64, vp, sz, vp]),
            ("mxfp4_abi_version", it, [])]:
        if not hasattr(lib, name):
            raise _error(f"the library lacks {name}: rebuild it (__graft_entry__.build())")
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    if lib.mxfp4_abi_version() != MXFP4_ABI_VERSION:
        raise _error(f"the library has MXFP4 ABI version {lib.mxfp4_abi_version()}, this binding "
                     f"expects {MXFP4_ABI_VERSION}: rebuild it (__graft_entry__.build())")


def _lib():
    from . import load_library
    return load_library()


def _check(rc):
    if rc != 0:
        raise _error(f"nvfp4 status {rc}: {_lib().nvfp4_status_string(rc).decode()}")


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


@dataclass
class MXTensor:
    """One copy on the GPU: codes uint8 [..., n, kp/2], scales uint8 [..., n, kp/32], where kp
    is k rounded up to a multiple of 128, or, for a grouped columnwise copy (n_groups > 0, k
    the number of grouped rows), mxfp4_grouped_k(k, n_groups)."""
    codes: torch.Tensor
    scales: torch.Tensor
    k: int
    n_groups: int = 0

    @property
    def shape(self):
        return (*self.codes.shape[:-1], self.k)

    def c(self):
        return MXTensorC(self.codes.data_ptr(), self.scales.data_ptr())

    @staticmethod
    def empty(n, k, device, n_groups=0):
        """Uninitialised copy; n: the number of rows, or a tuple (batch, rows)."""
        kp = grouped_k(k, n_groups) if n_groups else padded_k(k)
        n = n if isinstance(n, tuple) else (n,)
        return MXTensor(torch.empty((*n, kp // 2), dtype=torch.uint8, device=device),
                        torch.empty((*n, kp // 32), dtype=torch.uint8, device=device), k, n_groups)


def padded_k(k):
    """mxfp4_padded_k: the K extent of a copy's rows."""
    return (k + 127) // 128 * 128


def grouped_k(rows, n_groups):
    """mxfp4_grouped_k: the K extent of a grouped columnwise copy."""
    return (rows + min(rows, n_groups) * 127) // 128 * 128


def _operand(t, name, device=None):
    """Checks a copy's tensors; a kernel reads them by their extents alone."""
    codes, scales = t.codes, t.scales
    if not (codes.is_cuda and scales.is_cuda):
        raise _error("mxfp4 kernels take GPU tensors only (no CPU path)")
    kp = grouped_k(t.k, t.n_groups) if t.n_groups else padded_k(t.k)
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not codes.is_contiguous() \
            or not scales.is_contiguous():
        raise _error(f"{name}: codes and scales must be contiguous uint8 tensors")
    if codes.dim() < 2 or codes.shape[-1] * 2 != kp or scales.shape[-1] * 32 != kp \
            or codes.shape[:-1] != scales.shape[:-1]:
        raise _error(f"{name}: codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not "
                     f"hold rows of k = {t.k}")
    if scales.device != codes.device or (device is not None and codes.device != device):
        raise _error(f"{name} is on another device")
    return MXTensorC(codes.data_ptr(), scales.data_ptr())


def _groups(offsets, device):
    """(pointer, n_groups) of an offsets tensor; (None, 0) without one."""
    if offsets is None:
        return None, 0
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous() \
            or offsets.device != device or offsets.numel() < 2:
        raise _error("offsets must be a contiguous 1-D int32 tensor of n_groups + 1 >= 2 entries "
                     "on the operands' device")
    return offsets.data_ptr(), offsets.numel() - 1


def _matrix(x, name):
    if not x.is_cuda:
        raise _error("mxfp4 kernels take GPU tensors only (no CPU path)")
    if x.dtype not in _DTYPES:
        raise _error(f"unsupported dtype {x.dtype}")
    if x.shape[-1] > 1 and x.stride(-1) != 1:
        raise _error(f"{name} must have unit column stride")


def _pitch(x):
    """Row pitch of a matrix whose rows may be views of wider ones."""
    pitch, cols = x.stride(-2), x.shape[-1]
    if x.shape[-2] > 1 and pitch < cols:
        raise _error("rows overlap (row stride below the number of columns)")
    return max(pitch, cols)


def _output(out, shape, dtype, device):
    if out is None:
        if dtype not in _DTYPES:
            raise _error(f"unsupported dtype {dtype}")
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != tuple(shape) or out.device != device:
        raise _error(f"out must be a {tuple(shape)} tensor on the operands' device")
    _matrix(out, "out")
    return out


def mxfp4_quant_params(rowwise=True, colwise=False, scale_rule=MXFP4_SCALE_FLOOR, round_row=0,
                       round_col=0, seed=0):
    """Options of mxfp4_quantize; round_row, round_col: NVFP4_RNE (0) or NVFP4_SR (1)."""
    return MxQuantParams(int(rowwise), int(colwise), int(scale_rule), int(round_row), int(round_col),
                         int(seed) & 0xFFFFFFFFFFFFFFFF)


def mxfp4_quantize(x, params, offsets=None, row_out=None, col_out=None):
    """Quantize a bf16/fp32 CUDA tensor [rows][cols] or [batch][rows][cols] (any row and batch
    strides, unit column stride).  Returns (row_copy, col_copy), None for one not requested: the
    rowwise copy [.., rows][cols] and the columnwise copy [.., cols][rows].  With offsets (2-D x
    only) the columnwise copy's blocks restart at each group of rows."""
    _matrix(x, "x")
    if x.dim() not in (2, 3):
        raise _error("x must be a 2-D or 3-D tensor")
    dev = x.device
    op, groups = _groups(offsets, dev)
    if groups and x.dim() != 2:
        raise _error("grouped rows need a 2-D x")
    R, C = x.shape[-2:]
    batch = x.shape[0] if x.dim() == 3 else 1
    lead = (batch,) if x.dim() == 3 else ()
    row = col = None
    if params.rowwise:
        row = row_out if row_out is not None else MXTensor.empty((*lead, R), C, dev)
        rc = _operand(row, "row_out", dev)
        if row.shape != (*lead, R, C) or row.n_groups:
            raise _error(f"row_out {row.shape} does not hold x {tuple(x.shape)}")
    if params.colwise:
        col = col_out if col_out is not None else MXTensor.empty((*lead, C), R, dev, groups)
        cc = _operand(col, "col_out", dev)
        if col.shape != (*lead, C, R) or col.n_groups != groups:
            raise _error(f"col_out {col.shape} does not hold x {tuple(x.shape)} transposed")
    _check(_lib().mxfp4_quantize(x.data_ptr(), _DTYPES[x.dtype], batch, R, C, _pitch(x),
                                 x.stride(0) if batch > 1 else 0, op, groups, params,
                                 rc if row is not None else None, cc if col is not None else None,
                                 _stream(dev)))
    return row, col


def mxfp4_dequantize(q, out_dtype=torch.float32, offsets=None, out=None):
    """The values of a copy, [.., n][k]; a grouped columnwise copy takes its offsets."""
    qc = _operand(q, "q")
    dev = q.codes.device
    op, groups = _groups(offsets, dev)
    if groups != q.n_groups:
        raise _error(f"the copy has {q.n_groups} groups, offsets {groups}")
    out = _output(out, q.shape, out_dtype, dev)
    if out.dim() > 2 and not out.is_contiguous():
        raise _error("out of a stack of matrices must be contiguous")
    n = 1
    for d in q.codes.shape[:-1]:
        n *= d
    _check(_lib().mxfp4_dequantize(qc, n, q.k, op, groups, _DTYPES[out.dtype], out.data_ptr(),
                                   _pitch(out), _stream(dev)))
    return out


def mxfp4_gemm(a, b, out=None, out_dtype=torch.float32):
    """C = A B^T (A: M x K copy, B: N x K copy)."""
    ac = _operand(a, "a")
    dev = a.codes.device
    bc = _operand(b, "b", dev)
    if a.codes.dim() != 2 or b.codes.dim() != 2 or a.n_groups or b.n_groups:
        raise _error("mxfp4_gemm takes two plain copies")
    M, N = a.codes.shape[0], b.codes.shape[0]
    if a.k != b.k:
        raise _error(f"K mismatch {a.k} vs {b.k}")
    out = _output(out, (M, N), out_dtype, dev)
    _check(_lib().mxfp4_gemm(ac, bc, M, N, a.k, out.data_ptr(), _DTYPES[out.dtype], _pitch(out),
                             _stream(dev)))
    return out


def mxfp4_gemm_grouped(a, b, offsets, out=None, out_dtype=torch.float32):
    """C's rows of group g = A's rows of group g times B[g]^T (A: M x K copy, B: [n_groups] of
    N x K copies).  Rows in no group give 0."""
    ac = _operand(a, "a")
    dev = a.codes.device
    bc = _operand(b, "b", dev)
    op, groups = _groups(offsets, dev)
    if a.codes.dim() != 2 or b.codes.dim() != 3 or a.n_groups or b.n_groups:
        raise _error("mxfp4_gemm_grouped takes a copy of a matrix and one of a stack of matrices")
    if b.codes.shape[0] != groups:
        raise _error(f"{b.codes.shape[0]} matrices for {groups} groups")
    M, N = a.codes.shape[0], b.codes.shape[1]
    if a.k != b.k:
        raise _error(f"K mismatch {a.k} vs {b.k}")
    out = _output(out, (M, N), out_dtype, dev)
    _check(_lib().mxfp4_gemm_grouped(ac, bc, op, groups, M, N, a.k, out.data_ptr(),
                                     _DTYPES[out.dtype], _pitch(out), _stream(dev)))
    return out


def mxfp4_gemm_grouped_wgrad(a, b, offsets, out=None, out_dtype=torch.float32):
    """C[g] = A_g B_g^T over group g's span of two grouped columnwise copies (A: [M][rows],
    B: [N][rows]); returns [n_groups][M][N], 0 for an empty group."""
    ac = _operand(a, "a")
    dev = a.codes.device
    bc = _operand(b, "b", dev)
    op, groups = _groups(offsets, dev)
    if a.codes.dim() != 2 or b.codes.dim() != 2 or a.n_groups != groups or b.n_groups != groups:
        raise _error("mxfp4_gemm_grouped_wgrad takes two columnwise copies made with these offsets")
    if a.k != b.k:
        raise _error(f"row mismatch {a.k} vs {b.k}")
    M, N = a.codes.shape[0], b.codes.shape[0]
    out = _output(out, (groups, M, N), out_dtype, dev)
    if not out.is_contiguous():
        raise _error("out must be contiguous")
    _check(_lib().mxfp4_gemm_grouped_wgrad(ac, bc, op, groups, M, N, a.k, out.data_ptr(),
                                           _DTYPES[out.dtype], N, _stream(dev)))
    return out


def mxfp4_linear_workspace_bytes(M, N, K, n_groups=0):
    return int(_lib().mxfp4_linear_workspace_bytes(M, N, K, n_groups))


def mxfp4_linear(x, w, offsets=None, scale_rule=MXFP4_SCALE_FLOOR, out=None, out_dtype=None,
                 workspace=None):
    """Y = Q(x) W^T: x [M][K] bf16/fp32 is quantized rowwise on the way (w: N x K copy, or, with
    offsets, a stack of one per group).  out_dtype: x's unless given."""
    _matrix(x, "x")
    if x.dim() != 2:
        raise _error("x must be a 2-D tensor")
    dev = x.device
    wc = _operand(w, "w", dev)
    op, groups = _groups(offsets, dev)
    if w.codes.dim() != (3 if groups else 2) or w.n_groups or (groups and w.codes.shape[0] != groups):
        raise _error("w must be one copy, or with offsets a stack of one copy per group")
    M, K = x.shape
    N = w.codes.shape[-2]
    if w.k != K:
        raise _error(f"K mismatch {K} vs {w.k}")
    out = _output(out, (M, N), out_dtype or x.dtype, dev)
    lib = _lib()
    if workspace is None:
        need = lib.mxfp4_linear_workspace_bytes(M, N, K, groups)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise _error("workspace must be a contiguous uint8 tensor on x's device")
    ws, ws_bytes = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
    _check(lib.mxfp4_linear(x.data_ptr(), _DTYPES[x.dtype], M, K, _pitch(x), scale_rule, wc, N, op,
                            groups, out.data_ptr(), _DTYPES[out.dtype], _pitch(out), ws, ws_bytes,
                            _stream(dev)))
    return out
