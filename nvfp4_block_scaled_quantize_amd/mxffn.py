"""Binding of the gated feed-forward block and of the 8-bit activation checkpoints (C ABI in
``include/mxffn.h``, built into ``libnvfp4.so``).

  mxfp8_quantize         an MXFP8 checkpoint of a bf16/fp32 matrix or a stack of matrices: E4M3
                         elements, one E8M0 scale per 32, nothing saturates
  mxfp8_dequantize       its values
  mxfp8_to_mxfp4         rowwise and/or columnwise MXFP4 copies of its values
  mxfp4_gated            H = a(A Wg^T) (A Wu^T) over packed operands: as a tensor, as the packed
                         operand of the down projection, and with G and U kept as a checkpoint
  mxfp4_gated_linear     the same from activations in one call, for serving
  mxfp4_gated_backward   dH = dY W2, and with the checkpoint [dG dU] and H
  mxfp8_gated_backward   the same from dH

As in ``mxfp4.py`` this module only marshals arguments, and ``offsets`` groups rows by expert.
"""
import ctypes
import math

import torch

from . import mxfp4 as _mx
from .mxfp4 import MXFP4_SCALE_FLOOR, MXTensor, MXTensorC, MxQuantParams

MXFP4_SILU, MXFP4_GELU = 0, 1
MXFFN_ABI_VERSION = 1   # MXFFN_ABI_VERSION of include/mxffn.h this binding matches

MXFFN_EXPORTED = ["mxfp8_quantize", "mxfp8_dequantize", "mxfp8_to_mxfp4", "mxfp4_gated",
                  "mxfp4_gated_linear_workspace_bytes", "mxfp4_gated_linear", "mxfp4_gated_backward",
                  "mxfp8_gated_backward", "mxffn_abi_version"]

_error = _mx._error


def bind(lib):
    """Declares these functions' types on a loaded libnvfp4.so.  Returns what keeps this binding
    from using them, or None: the other calls need none of them."""
    lacking = [name for name in MXFFN_EXPORTED if not hasattr(lib, name)]
    if lacking:
        return f"the library lacks {lacking[0]}: rebuild it (__graft_entry__.build())"
    if lib.mxffn_abi_version() != MXFFN_ABI_VERSION:
        return (f"the library has MXFFN ABI version {lib.mxffn_abi_version()}, this binding expects "
                f"{MXFFN_ABI_VERSION}: rebuild it (__graft_entry__.build())")
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    it = ctypes.c_int
    T, Q = ctypes.POINTER(MXTensorC), ctypes.POINTER(MxQuantParams)    # a checkpoint's struct is laid out as a copy's
    for name, res, args in [
            ("mxfp8_quantize", it, [vp, it, i64, i64, i64, i64, i64, T, vp]),
            ("mxfp8_dequantize", it, [T, i64, i64, it, vp, i64, vp]),
            ("mxfp8_to_mxfp4", it, [T, i64, i64, i64, vp, i64, Q, T, T, vp]),
            ("mxfp4_gated", it, [T, T, vp, i64, i64, i64, i64, i32, vp, it, i64, i32, T, T, vp]),
            ("mxfp4_gated_linear_workspace_bytes", sz, [i64, i64, i64, i64]),
            ("mxfp4_gated_linear", it, [vp, it, i64, i64, i64, i32, T, i64, vp, i64, i32, vp, it, i64, vp, sz, vp]),
            ("mxfp4_gated_backward", it, [T, T, vp, i64, i64, i64, i64, i32, T, vp, it, i64, vp, i64, vp]),
            ("mxfp8_gated_backward", it, [vp, it, i64, i64, i64, i32, T, vp, it, i64, vp, i64, vp]),
            ("mxffn_abi_version", it, [])]:
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


class MX8Tensor:
    """One checkpoint on the GPU: codes uint8 [..., n, kp] (E4M3), scales uint8 [..., n, kp/32], where
    kp is k rounded up to a multiple of 128.  mxfp4_gated's holds G and U: [2, M, N].

    A checkpoint made by empty() or a call holds both in one buffer, codes first; codes and scales are
    views of it, made when they are asked for."""
    __slots__ = ("_codes", "_scales", "k", "_data", "_lead", "_rows")

    def __init__(self, codes, scales, k):
        self._codes, self._scales, self.k, self._data = codes, scales, k, None

    @staticmethod
    def empty(n, k, device):
        """Uninitialised checkpoint; n: the number of rows, or a tuple (batch, rows)."""
        return _new8(n if isinstance(n, tuple) else (n,), k, device)[0]

    def _views(self):
        kp = _mx.padded_k(self.k)
        split = self._rows * kp
        self._codes = self._data[:split].view(*self._lead, kp)
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
        return f"MX8Tensor(shape={self.shape}, device={_mx._held(self).device})"


def _new8(lead, k, device):
    """An uninitialised checkpoint and its C struct."""
    kp = (k + 127) // 128 * 128
    rows = lead[0] if len(lead) == 1 else math.prod(lead)
    split = rows * kp
    t = MX8Tensor(None, None, k)
    t._lead, t._rows = lead, rows
    t._data = torch.empty_strided((split + split // 32,), (1,), dtype=torch.uint8, device=device)
    at = t._data.data_ptr()
    return t, MXTensorC(at, at + split)


def _operand8(t, name, device):
    """Checks a checkpoint's tensors; returns them as the C struct and the extents before the last."""
    if not isinstance(t, MX8Tensor):
        raise _error(f"{name} must be an MX8Tensor")
    kp, data = (t.k + 127) // 128 * 128, t._data
    if data is not None:
        if data.get_device() != device:
            _mx._device(data)
            raise _error(f"{name} is on another device")
        split = t._rows * kp
        if data.numel() != split + split // 32:
            raise _error(f"{name}: its buffer does not hold rows of k = {t.k}")
        at = data.data_ptr()
        return MXTensorC(at, at + split), t._lead
    codes, scales = t.codes, t.scales
    if codes.get_device() != device or scales.get_device() != device:
        _mx._device(codes), _mx._device(scales)
        raise _error(f"{name} is on another device")
    *lead, width = codes.shape
    if not lead or width != kp or scales.shape != (*lead, kp // 32):
        raise _error(f"{name}: codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not "
                     f"hold rows of k = {t.k}")
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not codes.is_contiguous() \
            or not scales.is_contiguous():
        raise _error(f"{name}: codes and scales must be contiguous uint8 tensors")
    return MXTensorC(codes.data_ptr(), scales.data_ptr()), tuple(lead)


def _operand4(t, name, device):
    if not isinstance(t, MXTensor):
        raise _error(f"{name} must be an MXTensor")
    return _mx._operand(t, name, device)


def mxfp8_quantize(x, out=None):
    """An MXFP8 checkpoint of a bf16/fp32 CUDA tensor [rows][cols] or [batch][rows][cols] (any batch
    stride, rows that do not overlap, unit column stride)."""
    dev, shape, dtype, pitch = _mx._matrix(x, "x")
    if len(shape) > 3:
        raise _error("x must be a 2-D or 3-D tensor")
    rows, cols = shape[-2:]
    lead = tuple(shape[:-1])
    batch = lead[0] if len(lead) > 1 else 1
    if out is None:
        out, q = _new8(lead, cols, x.device)
    else:
        q, got = _operand8(out, "out", dev)
        if got != lead or out.k != cols:
            raise _error(f"out {out.shape} does not hold x {tuple(shape)}")
    _mx._call(_lib().mxfp8_quantize, dev, x.data_ptr(), dtype, batch, rows, cols, pitch,
              x.stride(0) if batch > 1 else 0, q)
    return out


def mxfp8_dequantize(q, out_dtype=torch.float32, out=None):
    """The values of a checkpoint, [.., n][k]."""
    held = _mx._held(q)
    dev = _mx._device(held)
    qc, lead = _operand8(q, "q", dev)
    out, dtype, pitch = _mx._output(out, (*lead, q.k), out_dtype, held)
    n = lead[0]
    if len(lead) > 1:
        if not out.is_contiguous():
            raise _error("out of a stack of matrices must be contiguous")
        # all its rows are one run; the stride of an axis of length 1 says nothing of them
        n, pitch = math.prod(lead), q.k
    _mx._call(_lib().mxfp8_dequantize, dev, qc, n, q.k, dtype, out.data_ptr(), pitch)
    return out


def mxfp8_to_mxfp4(q, params, offsets=None, row_out=None, col_out=None):
    """MXFP4 copies of a checkpoint's values, [rows][cols] or [batch][rows][cols]: returns (row_copy,
    col_copy) as mxfp4_quantize of mxfp8_dequantize(q, torch.bfloat16) would, bit for bit."""
    held = _mx._held(q)
    dev = _mx._device(held)
    qc, lead = _operand8(q, "q", dev)
    if len(lead) > 2:
        raise _error("q must hold a matrix or a stack of matrices")
    op, groups = _mx._groups(offsets, dev)
    if groups and len(lead) != 1:
        raise _error("grouped rows need a 2-D q")
    R, C = lead[-1], q.k
    batch = lead[0] if len(lead) > 1 else 1
    row, rc = _copy_out(row_out, "row_out", lead, C, 0, held) if params.rowwise else (None, None)
    col, cc = _copy_out(col_out, "col_out", (*lead[:-1], C), R, groups, held) if params.colwise else (None, None)
    _mx._call(_lib().mxfp8_to_mxfp4, dev, qc, batch, R, C, op, groups, params, rc, cc)
    return row, col


def _copy_out(given, name, lead, k, groups, like):
    """An MXFP4 copy to be written and its C struct: `given`, or a new one."""
    if given is None:
        return _mx._new(lead, k, like.device, groups)
    c, got = _operand4(given, name, like.get_device())
    if got != tuple(lead) or given.k != k or given.n_groups != groups:
        raise _error(f"{name} {given.shape} must be a copy of shape {(*lead, k)}")
    return given, c


def _weights(w, sw, groups, even):
    """Rows of each matrix of w, one per group where there are groups."""
    if len(sw) != (2 if groups else 1) or w.n_groups or (groups and sw[0] != groups):
        raise _error("w must be one copy, or with offsets a stack of one copy per group")
    if even and sw[-1] % 2:
        raise _error(f"w has {sw[-1]} rows: it must hold those of the gate and as many of the up projection")
    return sw[-1]


def mxfp4_gated(a, w, offsets=None, activation=MXFP4_SILU, out=None, out_dtype=torch.bfloat16, packed=False,
                scale_rule=MXFP4_SCALE_FLOOR, checkpoint=False):
    """H = a(A Wg^T) (A Wu^T) (A: M x K copy; w: 2N x K copy, the gate's rows first, or with offsets a
    stack of one per group).  Returns (h, h_copy, checkpoint), None for what is not asked for:
      h           a tensor of out_dtype (None: no tensor, unless `out` is given)
      h_copy      packed: True, or the MXTensor to fill: H's rowwise MXFP4 copy, rounded by scale_rule
      checkpoint  True, or the MX8Tensor to fill: [2, M, N], G and U"""
    held = _mx._held(a)
    dev = _mx._device(held)
    ac, sa = _operand4(a, "a", dev)
    wc, sw = _operand4(w, "w", dev)
    op, groups = _mx._groups(offsets, dev)
    if len(sa) != 1 or a.n_groups:
        raise _error("a must be a copy of a matrix")
    N = _weights(w, sw, groups, True) // 2
    if a.k != w.k:
        raise _error(f"K mismatch {a.k} vs {w.k}")
    M = sa[0]
    h = at = copy = qc = kept = kc = None
    dtype, pitch = 0, N
    if out is not None or out_dtype is not None:
        h, dtype, pitch = _mx._output(out, (M, N), out_dtype, held)
        at = h.data_ptr()
    if packed is not False and packed is not None:
        copy, qc = _copy_out(None if packed is True else packed, "packed", (M,), N, 0, held)
    if checkpoint is not False and checkpoint is not None:
        if checkpoint is True:
            kept, kc = _new8((2, M), N, held.device)
        else:
            kept = checkpoint
            kc, got = _operand8(kept, "checkpoint", dev)
            if got != (2, M) or kept.k != N:
                raise _error(f"checkpoint {kept.shape} must be of shape {(2, M, N)}")
    if h is None and copy is None and kept is None:
        raise _error("nothing to compute: a tensor, a packed copy or a checkpoint must be asked for")
    _mx._call(_lib().mxfp4_gated, dev, ac, wc, op, groups, M, N, a.k, activation, at, dtype, pitch, scale_rule, qc, kc)
    return h, copy, kept


def mxfp4_gated_linear_workspace_bytes(M, N, K, n_groups=0):
    return int(_lib().mxfp4_gated_linear_workspace_bytes(M, N, K, n_groups))


def mxfp4_gated_linear(x, w, offsets=None, activation=MXFP4_SILU, scale_rule=MXFP4_SCALE_FLOOR, out=None, out_dtype=None,
                       workspace=None):
    """H = a(Q(x) Wg^T) (Q(x) Wu^T): x [M][K] bf16/fp32 is quantized rowwise on the way (w: 2N x K copy, the
    gate's rows first, or with offsets a stack of one per group).  out_dtype: x's unless given."""
    dev, shape, xdtype, xpitch = _mx._matrix(x, "x")
    if len(shape) != 2:
        raise _error("x must be a 2-D tensor")
    wc, sw = _operand4(w, "w", dev)
    op, groups = _mx._groups(offsets, dev)
    M, K = shape
    N = _weights(w, sw, groups, True) // 2
    if w.k != K:
        raise _error(f"K mismatch {K} vs {w.k}")
    out, dtype, pitch = _mx._output(out, (M, N), out_dtype or x.dtype, x)
    lib = _lib()
    if workspace is None:
        need = lib.mxfp4_gated_linear_workspace_bytes(M, N, K, groups)
        workspace = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=x.device) if need else None
    elif workspace.get_device() != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise _error("workspace must be a contiguous uint8 tensor on x's device")
    ws, ws_bytes = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
    _mx._call(lib.mxfp4_gated_linear, dev, x.data_ptr(), xdtype, M, K, xpitch, scale_rule, wc, N, op, groups, activation,
              out.data_ptr(), dtype, pitch, ws, ws_bytes)
    return out


def _gradients(checkpoint, dev, out, out_dtype, h, like):
    """What both backward calls write: (M, N, checkpoint struct, dgu, dtype code, pitch, h, pointer, pitch)."""
    kc, lead = _operand8(checkpoint, "checkpoint", dev)
    if len(lead) != 2 or lead[0] != 2:
        raise _error(f"checkpoint {checkpoint.shape} must hold G and U: [2, M, N]")
    M, N = lead[1], checkpoint.k
    out, dtype, pitch = _mx._output(out, (M, 2 * N), out_dtype, like)
    at, ldh = None, N
    if h is False or h is None:
        h = None
    else:
        h, code, ldh = _mx._output(None if h is True else h, (M, N), out.dtype, like)
        if code != dtype:
            raise _error("h must be of the gradients' dtype")
        at = h.data_ptr()
    return M, N, kc, out, dtype, pitch, h, at, ldh


def mxfp4_gated_backward(dy, w, checkpoint, offsets=None, activation=MXFP4_SILU, out=None, out_dtype=torch.bfloat16, h=False):
    """dH = dY W2 (dy: dY's rowwise copy, M x K; w: W2's columnwise copy, N x K, or with offsets a stack of
    one per group), then with the checkpoint of mxfp4_gated ([2, M, N]) the gradients.  Returns (dgu,
    h): dgu [M][2N] holds dG and dU side by side; h is H = a(g) u where asked for (True, or the tensor to
    fill)."""
    held = _mx._held(dy)
    dev = _mx._device(held)
    ac, sa = _operand4(dy, "dy", dev)
    wc, sw = _operand4(w, "w", dev)
    op, groups = _mx._groups(offsets, dev)
    if len(sa) != 1 or dy.n_groups:
        raise _error("dy must be a copy of a matrix")
    rows = _weights(w, sw, groups, False)
    if dy.k != w.k:
        raise _error(f"K mismatch {dy.k} vs {w.k}")
    M, N, kc, out, dtype, pitch, h, at, ldh = _gradients(checkpoint, dev, out, out_dtype, h, held)
    if sa[0] != M or rows != N:
        raise _error(f"the checkpoint is of {M} x {N}, the product of {sa[0]} x {rows}")
    _mx._call(_lib().mxfp4_gated_backward, dev, ac, wc, op, groups, M, N, dy.k, activation, kc, out.data_ptr(), dtype, pitch,
              at, ldh)
    return out, h


def mxfp8_gated_backward(dh, checkpoint, activation=MXFP4_SILU, out=None, out_dtype=None, h=False):
    """The gradients of the gated product from dH [M][N] bf16/fp32 and the checkpoint ([2, M, N]).  Returns
    (dgu, h) as mxfp4_gated_backward; out_dtype: dh's unless given."""
    dev, shape, dhtype, dhpitch = _mx._matrix(dh, "dh")
    if len(shape) != 2:
        raise _error("dh must be a 2-D tensor")
    M, N, kc, out, dtype, pitch, h, at, ldh = _gradients(checkpoint, dev, out, out_dtype or dh.dtype, h, dh)
    if tuple(shape) != (M, N):
        raise _error(f"the checkpoint is of {M} x {N}, dh of {tuple(shape)}")
    _mx._call(_lib().mxfp8_gated_backward, dev, dh.data_ptr(), dhtype, dhpitch, M, N, activation, kc, out.data_ptr(), dtype,
              pitch, at, ldh)
    return out, h
