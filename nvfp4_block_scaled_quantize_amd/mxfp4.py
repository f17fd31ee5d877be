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
import math

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
    """Declares the MXFP4 functions' types on a loaded libnvfp4.so.  Returns what keeps this
    binding from using them, or None: the NVFP4 calls need none of them."""
    lacking = [name for name in MXFP4_EXPORTED if not hasattr(lib, name)]
    if lacking:
        return f"the library lacks {lacking[0]}: rebuild it (__graft_entry__.build())"
    if lib.mxfp4_abi_version() != MXFP4_ABI_VERSION:
        return (f"the library has MXFP4 ABI version {lib.mxfp4_abi_version()}, this binding expects "
                f"{MXFP4_ABI_VERSION}: rebuild it (__graft_entry__.build())")
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
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return None


_bound = None      # the package's library once it is loaded and these calls can use it
_unusable = None   # or why they cannot


def attach(lib, unusable):
    """Takes the package's library, with what bind() said of it."""
    global _bound, _unusable
    _bound, _unusable = (None if unusable else lib), unusable


def _lib():
    if _bound is None:
        from . import load_library
        load_library()
        if _bound is None:
            raise _error(_unusable)
    return _bound


# The current stream's handle by device index: a call of these operators can be shorter than
# building the torch.cuda.Stream object that would otherwise carry it (0.1 against 1.9 us).
_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice


def _call(f, device, *args):
    """f(*args, stream) on the tensors' device, which need not be the current one."""
    if _current() == device:
        rc = f(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            rc = f(*args, _stream(device))
    if rc != 0:
        raise _error(f"nvfp4 status {rc}: {_lib().nvfp4_status_string(rc).decode()}")


class MXTensor:
    """One copy on the GPU: codes uint8 [..., n, kp/2], scales uint8 [..., n, kp/32], where kp
    is k rounded up to a multiple of 128, or, for a grouped columnwise copy (n_groups > 0, k
    the number of grouped rows), mxfp4_grouped_k(k, n_groups).

    A copy made by empty() or mxfp4_quantize holds both in one buffer, codes first; codes and
    scales are views of it, made when they are asked for (a call of these operators can be
    shorter than an allocation and two views)."""
    __slots__ = ("_codes", "_scales", "k", "n_groups", "_data", "_lead", "_rows")

    def __init__(self, codes, scales, k, n_groups=0):
        self._codes, self._scales, self.k, self.n_groups, self._data = codes, scales, k, n_groups, None

    @staticmethod
    def empty(n, k, device, n_groups=0):
        """Uninitialised copy; n: the number of rows, or a tuple (batch, rows)."""
        return _new(n if isinstance(n, tuple) else (n,), k, device, n_groups)[0]

    def _views(self):
        kp = grouped_k(self.k, self.n_groups) if self.n_groups else padded_k(self.k)
        split = self._rows * (kp // 2)
        self._codes = self._data[:split].view(*self._lead, kp // 2)
        self._scales = self._data[split:].view(*self._lead, kp // 32)

    @property
    def codes(self):
        if self._codes is None:
            self._views()
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._views()
        return self._scales

    @codes.setter
    def codes(self, value):
        self._scales, self._codes, self._data = self.scales, value, None

    @scales.setter
    def scales(self, value):
        self._codes, self._scales, self._data = self.codes, value, None

    @property
    def shape(self):
        return (*(self.codes.shape[:-1] if self._data is None else self._lead), self.k)

    def __repr__(self):
        return f"MXTensor(shape={self.shape}, n_groups={self.n_groups}, device={_held(self).device})"


def _new(lead, k, device, n_groups):
    """An uninitialised copy and its C struct."""
    kp = grouped_k(k, n_groups) if n_groups else (k + 127) // 128 * 128
    rows = lead[0] if len(lead) == 1 else math.prod(lead)
    split = rows * (kp // 2)
    t = MXTensor(None, None, k, n_groups)
    t._lead, t._rows = lead, rows
    t._data = torch.empty_strided((split + split // 16,), (1,), dtype=torch.uint8, device=device)
    at = t._data.data_ptr()
    return t, MXTensorC(at, at + split)


def _held(t):
    """A tensor of the copy's memory."""
    return t.codes if t._data is None else t._data


def padded_k(k):
    """mxfp4_padded_k: the K extent of a copy's rows."""
    return (k + 127) // 128 * 128


def grouped_k(rows, n_groups):
    """mxfp4_grouped_k: the K extent of a grouped columnwise copy."""
    return (rows + min(rows, n_groups) * 127) // 128 * 128


def _device(t):
    """Device index of a CUDA tensor."""
    d = t.get_device()
    if d < 0:
        raise _error("mxfp4 kernels take GPU tensors only (no CPU path)")
    return d


def _operand(t, name, device):
    """Checks a copy's tensors (a kernel reads them by their extents alone); returns them as the
    C struct and the extents before the last."""
    data, k = t._data, t.k
    kp = (k + 127) // 128 * 128 if not t.n_groups else grouped_k(k, t.n_groups)
    if data is not None:
        if data.get_device() != device:
            _device(data)
            raise _error(f"{name} is on another device")
        split = t._rows * (kp // 2)
        if data.numel() != split + split // 16:
            raise _error(f"{name}: its buffer does not hold rows of k = {k}")
        at = data.data_ptr()
        return MXTensorC(at, at + split), t._lead
    codes, scales = t.codes, t.scales
    if codes.get_device() != device or scales.get_device() != device:
        _device(codes), _device(scales)
        raise _error(f"{name} is on another device")
    *lead, width = codes.shape
    if not lead or width * 2 != kp or scales.shape != (*lead, kp // 32):
        raise _error(f"{name}: codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not "
                     f"hold rows of k = {k}")
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not codes.is_contiguous() \
            or not scales.is_contiguous():
        raise _error(f"{name}: codes and scales must be contiguous uint8 tensors")
    return MXTensorC(codes.data_ptr(), scales.data_ptr()), tuple(lead)


def _groups(offsets, device):
    """(pointer, n_groups) of an offsets tensor; (None, 0) without one."""
    if offsets is None:
        return None, 0
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous() \
            or offsets.get_device() != device or offsets.numel() < 2:
        raise _error("offsets must be a contiguous 1-D int32 tensor of n_groups + 1 >= 2 entries "
                     "on the operands' device")
    return offsets.data_ptr(), offsets.numel() - 1


def _matrix(x, name):
    """(device index, shape, dtype code, row pitch) of a matrix or a stack of them whose rows
    may be views of wider ones."""
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise _error(f"unsupported dtype {x.dtype}")
    device, shape = _device(x), x.shape
    if len(shape) == 2:
        (rows, cols), (pitch, step) = shape, x.stride()
    elif len(shape) < 2:
        raise _error(f"{name} must be a matrix")
    else:
        (rows, cols), (pitch, step) = shape[-2:], x.stride()[-2:]
    if cols > 1 and step != 1:
        raise _error(f"{name} must have unit column stride")
    if pitch < cols:
        if rows > 1:
            raise _error(f"{name}'s rows overlap (row stride below the number of columns)")
        pitch = cols
    return device, shape, dtype, pitch


def _output(out, shape, dtype, like):
    """(out, dtype code, row pitch), allocated on `like`'s device unless given."""
    if out is None:
        code = _DTYPES.get(dtype)
        if code is None:
            raise _error(f"unsupported dtype {dtype}")
        if len(shape) == 2:     # empty_strided takes 0.4 us less than empty
            out = torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=like.device)
        else:
            out = torch.empty(shape, dtype=dtype, device=like.device)
        return out, code, shape[-1]
    device, got, code, pitch = _matrix(out, "out")
    if got != shape or device != like.get_device():
        raise _error(f"out must be a {shape} tensor on the operands' device")
    return out, code, pitch


def mxfp4_quant_params(rowwise=True, colwise=False, scale_rule=MXFP4_SCALE_FLOOR, round_row=0,
                       round_col=0, seed=0):
    """Options of mxfp4_quantize; round_row, round_col: NVFP4_RNE (0) or NVFP4_SR (1)."""
    return MxQuantParams(int(rowwise), int(colwise), int(scale_rule), int(round_row), int(round_col),
                         int(seed) & 0xFFFFFFFFFFFFFFFF)


def mxfp4_quantize(x, params, offsets=None, row_out=None, col_out=None):
    """Quantize a bf16/fp32 CUDA tensor [rows][cols] or [batch][rows][cols] (any batch stride, rows
    that do not overlap, unit column stride).  Returns (row_copy, col_copy), None for one not
    requested: the rowwise copy [.., rows][cols] and the columnwise copy [.., cols][rows].  With
    offsets (2-D x only) the columnwise copy's blocks restart at each group of rows."""
    dev, shape, dtype, pitch = _matrix(x, "x")
    if len(shape) > 3:
        raise _error("x must be a 2-D or 3-D tensor")
    op, groups = _groups(offsets, dev)
    if groups and len(shape) != 2:
        raise _error("grouped rows need a 2-D x")
    R, C = shape[-2:]
    lead = tuple(shape[:-2])
    batch = lead[0] if lead else 1
    row = col = rc = cc = None
    if params.rowwise:
        if row_out is None:
            row, rc = _new((*lead, R), C, x.device, 0)
        else:
            row = row_out
            rc, got = _operand(row, "row_out", dev)
            if got != (*lead, R) or row.k != C or row.n_groups:
                raise _error(f"row_out {row.shape} does not hold x {tuple(shape)}")
    if params.colwise:
        if col_out is None:
            col, cc = _new((*lead, C), R, x.device, groups)
        else:
            col = col_out
            cc, got = _operand(col, "col_out", dev)
            if got != (*lead, C) or col.k != R or col.n_groups != groups:
                raise _error(f"col_out {col.shape} does not hold x {tuple(shape)} transposed")
    _call(_lib().mxfp4_quantize, dev, x.data_ptr(), dtype, batch, R, C, pitch,
          x.stride(0) if batch > 1 else 0, op, groups, params, rc, cc)
    return row, col


def mxfp4_dequantize(q, out_dtype=torch.float32, offsets=None, out=None):
    """The values of a copy, [.., n][k]; a grouped columnwise copy takes its offsets."""
    held = _held(q)
    dev = _device(held)
    qc, lead = _operand(q, "q", dev)
    op, groups = _groups(offsets, dev)
    if groups != q.n_groups:
        raise _error(f"the copy has {q.n_groups} groups, offsets {groups}")
    out, dtype, pitch = _output(out, (*lead, q.k), out_dtype, held)
    n = lead[0]
    if len(lead) > 1:
        if not out.is_contiguous():
            raise _error("out of a stack of matrices must be contiguous")
        # all its rows are one run; the stride of an axis of length 1 says nothing of them
        n, pitch = math.prod(lead), q.k
    _call(_lib().mxfp4_dequantize, dev, qc, n, q.k, op, groups, dtype, out.data_ptr(), pitch)
    return out


def mxfp4_gemm(a, b, out=None, out_dtype=torch.float32):
    """C = A B^T (A: M x K copy, B: N x K copy)."""
    held = _held(a)
    dev = _device(held)
    ac, sa = _operand(a, "a", dev)
    bc, sb = _operand(b, "b", dev)
    if len(sa) != 1 or len(sb) != 1 or a.n_groups or b.n_groups:
        raise _error("mxfp4_gemm takes two plain copies")
    if a.k != b.k:
        raise _error(f"K mismatch {a.k} vs {b.k}")
    M, N = sa[0], sb[0]
    out, dtype, pitch = _output(out, (M, N), out_dtype, held)
    _call(_lib().mxfp4_gemm, dev, ac, bc, M, N, a.k, out.data_ptr(), dtype, pitch)
    return out


def mxfp4_gemm_grouped(a, b, offsets, out=None, out_dtype=torch.float32):
    """C's rows of group g = A's rows of group g times B[g]^T (A: M x K copy, B: [n_groups] of
    N x K copies).  Rows in no group give 0."""
    held = _held(a)
    dev = _device(held)
    ac, sa = _operand(a, "a", dev)
    bc, sb = _operand(b, "b", dev)
    op, groups = _groups(offsets, dev)
    if len(sa) != 1 or len(sb) != 2 or a.n_groups or b.n_groups:
        raise _error("mxfp4_gemm_grouped takes a copy of a matrix and one of a stack of matrices")
    if sb[0] != groups:
        raise _error(f"{sb[0]} matrices for {groups} groups")
    if a.k != b.k:
        raise _error(f"K mismatch {a.k} vs {b.k}")
    M, N = sa[0], sb[1]
    out, dtype, pitch = _output(out, (M, N), out_dtype, held)
    _call(_lib().mxfp4_gemm_grouped, dev, ac, bc, op, groups, M, N, a.k, out.data_ptr(), dtype, pitch)
    return out


def mxfp4_gemm_grouped_wgrad(a, b, offsets, out=None, out_dtype=torch.float32):
    """C[g] = A_g B_g^T over group g's span of two grouped columnwise copies (A: [M][rows],
    B: [N][rows]); returns [n_groups][M][N], 0 for an empty group."""
    held = _held(a)
    dev = _device(held)
    ac, sa = _operand(a, "a", dev)
    bc, sb = _operand(b, "b", dev)
    op, groups = _groups(offsets, dev)
    if len(sa) != 1 or len(sb) != 1 or a.n_groups != groups or b.n_groups != groups or not groups:
        raise _error("mxfp4_gemm_grouped_wgrad takes two columnwise copies made with these offsets")
    if a.k != b.k:
        raise _error(f"row mismatch {a.k} vs {b.k}")
    M, N = sa[0], sb[0]
    out, dtype, _ = _output(out, (groups, M, N), out_dtype, held)
    if not out.is_contiguous():
        raise _error("out must be contiguous")
    _call(_lib().mxfp4_gemm_grouped_wgrad, dev, ac, bc, op, groups, M, N, a.k, out.data_ptr(), dtype, N)
    return out


def mxfp4_linear_workspace_bytes(M, N, K, n_groups=0):
    return int(_lib().mxfp4_linear_workspace_bytes(M, N, K, n_groups))


def mxfp4_linear(x, w, offsets=None, scale_rule=MXFP4_SCALE_FLOOR, out=None, out_dtype=None,
                 workspace=None):
    """Y = Q(x) W^T: x [M][K] bf16/fp32 is quantized rowwise on the way (w: N x K copy, or, with
    offsets, a stack of one per group).  out_dtype: x's unless given."""
    dev, shape, xdtype, xpitch = _matrix(x, "x")
    if len(shape) != 2:
        raise _error("x must be a 2-D tensor")
    wc, sw = _operand(w, "w", dev)
    op, groups = _groups(offsets, dev)
    if len(sw) != (2 if groups else 1) or w.n_groups or (groups and sw[0] != groups):
        raise _error("w must be one copy, or with offsets a stack of one copy per group")
    M, K = shape
    N = sw[-1]
    if w.k != K:
        raise _error(f"K mismatch {K} vs {w.k}")
    out, dtype, pitch = _output(out, (M, N), out_dtype or x.dtype, x)
    lib = _lib()
    if workspace is None:
        need = lib.mxfp4_linear_workspace_bytes(M, N, K, groups)
        workspace = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=x.device) if need else None
    elif workspace.get_device() != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise _error("workspace must be a contiguous uint8 tensor on x's device")
    ws, ws_bytes = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
    _call(lib.mxfp4_linear, dev, x.data_ptr(), xdtype, M, K, xpitch, scale_rule, wc, N, op, groups,
          out.data_ptr(), dtype, pitch, ws, ws_bytes)
    return out
