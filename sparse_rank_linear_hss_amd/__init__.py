"""Sparse + low-rank (HSS) linear layer on AMD MI355X.

Thin Python binding of libhss.so (C ABI in include/hss.h).  The functions keep
the C names; they only marshal torch tensors (device memory) and the current
HIP stream into the C calls -- every step runs in the library's HIP kernels.

    W ~= S + U V^T,   Y = X (S + U V^T)^T

    sp = hss_split(W, "csr", frac=(5, 100), residual=True)   # stage 1 on the GPU
    A  = HSSMatrix.from_split(sp, U, V=V)                     # U: m x r, V: n x r
    Y  = hss_apply(A, X)                                      # X: b x n -> Y: b x m
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass, field
from typing import Optional

import torch

from ._lib import (HSS_BF16, HSS_COL16, HSS_DQ4, HSS_ERR_NONFINITE, HSS_HIER2, HSS_F32, HSS_FMT_2OF4, HSS_FMT_CSR,
                   HSS_MAX_BATCH, HSS_MX4, HSS_MX4_T, HSS_MX_GROUP, HSS_MXFP4, HSS_MXINT8, HSS_OK, HSS_OPT_BATCH_ROUTE, HSS_OPT_DECODE_FORCE_LOCAL, HSS_OPT_DECODE_MERGED,
                   HSS_OPT_DECODE_RPW, HSS_OPT_DECODE_WAVE_PRODUCERS,
                   HSS_OPT_DECODE_SPIN, HSS_OPT_GRAD_DS_ROUTE, HSSError, HssMatrixStruct, LIB_PATH, check, lib,
                   status_string)

__all__ = [
    "hss_version", "hss_topk_count", "hss_split_workspace_size", "hss_split", "hss_get_error",
    "hss_set_option", "hss_get_option", "option", "HSS_MAX_BATCH",
    "hss_apply_workspace_size", "hss_apply_workspace_init", "apply_workspace", "hss_apply", "hss_apply_noalloc",
    "hss_apply_group_workspace_size", "hss_apply_group",
    "hss_csr_cols_to_u16", "HSS_COL16", "HSS_DQ4", "HSS_HIER2",
    "hss_rcm_order", "hss_concentration", "hss_hier_pack", "hss_hier_pack_compact", "hss_csr_permute",
    "hss_grad", "hss_csr_transpose", "hss_gather_values", "hss_transpose", "hss_transposed_layer", "hss_backward",
    "hss_nm24_to_csr",
    "HSS_MX4", "HSS_MX4_T", "HSS_MX_GROUP", "MXTensor", "hss_mx_quantize", "hss_mx_dequantize",
    "hss_grad_ckpt", "hss_grad_ckpt_workspace_size", "grad_ckpt_workspace",
    "HSSMatrix", "SplitResult", "HSSError",
    "LIB_PATH", "status_string",
]

_DT = {torch.float32: HSS_F32, torch.bfloat16: HSS_BF16}
_FMT = {"csr": HSS_FMT_CSR, "2:4": HSS_FMT_2OF4, HSS_FMT_CSR: HSS_FMT_CSR, HSS_FMT_2OF4: HSS_FMT_2OF4}


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")
    return _DT[t.dtype]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    device = device if isinstance(device, torch.device) else torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"expected a GPU device, got {device}")
    return _raw_stream(torch.cuda.current_device() if device.index is None else device.index)


# A decode call is bound by its host side (4096 x 4096, one column: the launch
# itself takes 3.5 us), so the calls below read the handles that torch.cuda's
# own functions wrap, and make X's device current only where it is not: a launch
# goes to the current device.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _index(t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError("tensor must be on a GPU device")
    return index


def _on(t: torch.Tensor):
    """Scope with t's GPU current (nothing to do where it is, or for a CPU tensor, which the call then refuses)."""
    index = t.get_device()
    return contextlib.nullcontext() if index < 0 or index == _current_device() else torch.cuda.device(index)


def _dev(t: torch.Tensor):
    if not t.is_cuda:
        raise ValueError("tensor must be on a GPU device")
    return t.device


def hss_version() -> int:
    return lib.hss_version()


# Diagnostic switches (hss_set_option); route names as the environment
# variables spell them.
_OPTS = {"batch_route": HSS_OPT_BATCH_ROUTE, "grad_ds_route": HSS_OPT_GRAD_DS_ROUTE,
         "decode_spin": HSS_OPT_DECODE_SPIN, "decode_merged": HSS_OPT_DECODE_MERGED,
         "decode_force_local": HSS_OPT_DECODE_FORCE_LOCAL, "decode_wave_producers": HSS_OPT_DECODE_WAVE_PRODUCERS,
         "decode_rpw": HSS_OPT_DECODE_RPW}
_OPT_WORDS = {"batch_route": {"auto": 0, "decode": 1, "spmm": 2, "densify": 3, "smfmac": 4},
              "grad_ds_route": {"auto": 0, "sparse": 1, "dense": 2}}


def hss_set_option(name: str, value) -> None:
    """Set a process-wide diagnostic switch: batch_route (auto | decode | spmm |
    densify | smfmac), grad_ds_route (auto | sparse | dense), decode_spin
    (int), decode_merged (0 | 1), decode_force_local (0 | 1)."""
    v = _OPT_WORDS.get(name, {}).get(value, value)
    check(lib.hss_set_option(_OPTS[name], int(v)), f"hss_set_option({name})")


def hss_get_option(name: str) -> int:
    return int(lib.hss_get_option(_OPTS[name]))


@contextlib.contextmanager
def option(name: str, value):
    """Scope a diagnostic switch: set on entry, the previous value restored on exit."""
    old = hss_get_option(name)
    hss_set_option(name, value)
    try:
        yield
    finally:
        check(lib.hss_set_option(_OPTS[name], old), f"hss_set_option({name})")


def hss_topk_count(m: int, n: int, num: int, den: int) -> int:
    """floor(m*n*num/den) computed exactly by the library."""
    k = lib.hss_topk_count(m, n, num, den)
    if k < 0:
        raise ValueError("invalid count arguments")
    return int(k)


def hss_split_workspace_size(fmt, dtype: int, m: int, n: int) -> int:
    out = ctypes.c_size_t(0)
    check(lib.hss_split_workspace_size(_FMT[fmt], dtype, m, n, ctypes.byref(out)), "hss_split_workspace_size")
    return int(out.value)


@dataclass
class SplitResult:
    fmt: int
    m: int
    n: int
    k: int
    row_ptr: Optional[torch.Tensor] = None    # int32 [m+1]
    col_idx: Optional[torch.Tensor] = None    # int32 [k]
    values: Optional[torch.Tensor] = None     # W dtype [k]
    nm_values: Optional[torch.Tensor] = None  # W dtype [m, n/2]
    nm_meta: Optional[torch.Tensor] = None    # int32 storage of uint32 [m, ceil(n/32)]
    residual: Optional[torch.Tensor] = None   # W dtype [m, n]
    ws: Optional[torch.Tensor] = field(default=None, repr=False)


def hss_split(W: torch.Tensor, fmt="csr", k: Optional[int] = None, frac=(5, 100),
              residual: bool = False, check_finite: bool = True) -> SplitResult:
    """Stage 1 on the GPU: magnitude top-k of W (m x n) into CSR or 2:4.

    fmt "csr": k defaults to floor(m*n*frac[0]/frac[1]).  fmt "2:4": k is m*n/2.
    check_finite synchronises and raises HSSError(HSS_ERR_NONFINITE) on NaN/Inf."""
    dev = _dev(W)
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D tensor")
    dt = _dt(W)
    m, n = W.shape
    f = _FMT[fmt]
    ws_bytes = hss_split_workspace_size(f, dt, m, n)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    res = torch.empty_like(W) if residual else None
    out = SplitResult(fmt=f, m=m, n=n, k=0, residual=res, ws=ws)
    if f == HSS_FMT_CSR:
        if k is None:
            k = hss_topk_count(m, n, *frac)
        out.k = int(k)
        out.row_ptr = torch.empty(m + 1, dtype=torch.int32, device=dev)
        out.col_idx = torch.empty(max(out.k, 0), dtype=torch.int32, device=dev)
        out.values = torch.empty(max(out.k, 0), dtype=W.dtype, device=dev)
        with _on(W):
            code = lib.hss_split(f, dt, m, n, _ptr(W), out.k, _ptr(out.row_ptr),
                                 _ptr(out.col_idx) if out.k > 0 else None,
                                 _ptr(out.values) if out.k > 0 else None, None, None, _ptr(res),
                                 _ptr(ws), ws_bytes, _stream(dev))
    else:
        out.k = (m * n) // 2 if k is None else int(k)
        out.nm_values = torch.empty((m, n // 2), dtype=W.dtype, device=dev)
        out.nm_meta = torch.empty((m, (n + 31) // 32), dtype=torch.int32, device=dev)
        with _on(W):
            code = lib.hss_split(f, dt, m, n, _ptr(W), out.k, None, None, None, _ptr(out.nm_values),
                                 _ptr(out.nm_meta), _ptr(res), _ptr(ws), ws_bytes, _stream(dev))
    check(code, "hss_split")
    if check_finite:
        check(hss_get_error(ws), "hss_split")
    return out


def hss_get_error(ws: torch.Tensor) -> int:
    """Synchronises the current stream and returns the split's device status code."""
    return int(lib.hss_get_error(_ptr(ws), _stream(ws.device)))


# ---------------------------------------------------------------------------
# Microscaled formats
# ---------------------------------------------------------------------------

_MX_FMT = {"fp4": HSS_MXFP4, "int8": HSS_MXINT8}


class MXTensor:
    """A rows x cols matrix in a microscaled format: groups of 32 columns of a
    row share a power-of-two scale (the layout of hss_mx_quantize).

    fmt "fp4": codes uint8 [rows, 16 ng] (two 4-bit codes per byte); "int8":
    codes int8 [rows, 32 ng]; scales uint8 [rows, ng], ng = ceil(cols / 32)."""

    __slots__ = ("fmt", "rows", "cols", "codes", "scales", "index")

    def __init__(self, fmt, rows, cols, codes, scales):
        if fmt not in _MX_FMT:
            raise ValueError(f"unknown microscaled format {fmt!r}: 'fp4' or 'int8'")
        rows, cols = int(rows), int(cols)
        ng = -(-cols // HSS_MX_GROUP)
        want = (rows, 16 * ng) if fmt == "fp4" else (rows, 32 * ng)
        if codes.dtype != (torch.uint8 if fmt == "fp4" else torch.int8) or codes.shape != want or \
                not codes.is_contiguous():
            raise ValueError(f"codes of a {rows} x {cols} {fmt} matrix: contiguous "
                             f"{'uint8' if fmt == 'fp4' else 'int8'} {want}")
        if scales.dtype != torch.uint8 or scales.shape != (rows, ng) or not scales.is_contiguous():
            raise ValueError(f"scales of a {rows} x {cols} matrix: contiguous uint8 {(rows, ng)}")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        self.fmt, self.rows, self.cols, self.codes, self.scales = fmt, rows, cols, codes, scales
        self.index = codes.get_device()

    @classmethod
    def empty(cls, fmt, rows, cols, device):
        """Unwritten arrays, for hss_mx_quantize(..., out=)."""
        ng = -(-int(cols) // HSS_MX_GROUP)
        codes = torch.empty((rows, 16 * ng), dtype=torch.uint8, device=device) if fmt == "fp4" else \
            torch.empty((rows, 32 * ng), dtype=torch.int8, device=device)
        return cls(fmt, rows, cols, codes, torch.empty((rows, ng), dtype=torch.uint8, device=device))

    @property
    def device(self):
        return self.codes.device


def hss_mx_quantize(W: torch.Tensor, fmt="fp4", out: Optional[MXTensor] = None, residual=None):
    """W (rows x cols, fp32 or bf16) in a microscaled format: "fp4" (weights)
    or "int8" (activation checkpoints), each value within half a step.

    residual=True (or a tensor of W's shape and dtype, which may be W itself)
    also writes W minus the quantised values (exact) and returns (q, residual)."""
    index = _index(W)
    if index != _current_device():
        with torch.cuda.device(index):
            return hss_mx_quantize(W, fmt, out, residual)
    shape = W.shape
    if len(shape) != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D tensor")
    rows, cols = shape
    if out is None:
        out = MXTensor.empty(fmt, rows, cols, W.device)
    elif out.fmt != fmt or out.rows != rows or out.cols != cols or out.index != index:
        raise ValueError(f"out must be a {rows} x {cols} {fmt} MXTensor on {W.device}")
    res = None
    if residual is not False and residual is not None:
        res = torch.empty_like(W) if residual is True else residual
        if res.shape != shape or res.dtype != W.dtype or not res.is_contiguous() or res.get_device() != index:
            raise ValueError("residual must be a contiguous tensor of W's shape, dtype and device")
    code = lib.hss_mx_quantize(_MX_FMT[fmt], _dt(W), rows, cols, W.data_ptr(), out.codes.data_ptr(),
                               out.scales.data_ptr(), None if res is None else res.data_ptr(), _raw_stream(index))
    if code:
        check(code, "hss_mx_quantize")
    return out if res is None else (out, res)


def hss_mx_dequantize(q: MXTensor, dtype=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values q stands for (rows x cols, bf16 by default or fp32; exact in both)."""
    index = _index(q.codes)
    if index != _current_device():
        with torch.cuda.device(index):
            return hss_mx_dequantize(q, dtype, out)
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=dtype or torch.bfloat16, device=q.device)
    elif out.shape != (q.rows, q.cols) or not out.is_contiguous() or out.get_device() != index or \
            (dtype is not None and out.dtype != dtype):
        raise ValueError("out must be a contiguous tensor of q's shape and device")
    code = lib.hss_mx_dequantize(_MX_FMT[q.fmt], _dt(out), q.rows, q.cols, q.codes.data_ptr(), q.scales.data_ptr(),
                                 out.data_ptr(), _raw_stream(index))
    if code:
        check(code, "hss_mx_dequantize")
    return out


class HSSMatrix:
    """Compressed matrix S + U V^T (or S + D) in device memory; keeps its tensors alive.

    U: m x r row-major.  The factor V (n x r) is held as Vt (r x n row-major,
    i.e. V column-major), the layout the library reads.  CSR col_idx is
    int32, or 16-bit (a torch.int16 tensor holding the uint16 columns, n <=
    65536, see hss_csr_cols_to_u16) -- the matrix then carries HSS_COL16.
    dq_codes (uint8, m x n/2: the 4-bit codes of columns 2j and 2j+1 in the
    low and high nibble of byte j) with dq_levels (m x 16, the matrix dtype)
    add the quantised dense part D of the dense-and-sparse form (HSS_DQ4).
    hier_r (ranks of the 2 x 2 blocks 00, 01, 10, 11) makes the low-rank term
    the compact block form (HSS_HIER2): U m x (hier_r[0] + hier_r[1]) and
    Vt sum(hier_r) x (n - n // 2) as hss_hier_pack_compact writes them, the
    matrix in the blocks' (permuted) order.
    mx (an "fp4" MXTensor, m x n) adds a microscaled 4-bit dense part (HSS_MX4),
    next to S and the low-rank term; mx_t=True: mx holds its transpose, n x m
    (HSS_MX4_T).  row_ptr may then be left out for an empty S."""

    def __init__(self, fmt, m, n, dtype, U=None, Vt=None, row_ptr=None, col_idx=None, values=None,
                 nnz=None, nm_values=None, nm_meta=None, dq_codes=None, dq_levels=None, hier_r=None,
                 mx=None, mx_t=False):
        self.fmt = _FMT[fmt]
        self.flags = HSS_COL16 if (col_idx is not None and col_idx.dtype == torch.int16) else 0
        self.hier_r = None if hier_r is None else [int(v) for v in hier_r]
        if dq_codes is not None:
            assert dq_codes.dtype == torch.uint8 and dq_codes.is_contiguous() and dq_codes.numel() == m * n // 2
            assert dq_levels is not None and dq_levels.dtype == dtype and dq_levels.is_contiguous()
            assert dq_levels.numel() == m * 16
            self.flags |= HSS_DQ4
        self.dq_codes, self.dq_levels = dq_codes, dq_levels
        self.mx, self.mx_t = mx, bool(mx_t)
        if mx is not None:
            if dq_codes is not None:
                raise ValueError("one dense part: dq_codes or mx")
            if mx.fmt != "fp4" or (mx.rows, mx.cols) != ((n, m) if mx_t else (m, n)):
                raise ValueError(f"mx must be an 'fp4' MXTensor, {'n x m' if mx_t else 'm x n'} of the {m} x {n} matrix")
            if any(t is not None and t.device != mx.device for t in (U, Vt, row_ptr, col_idx, values)):
                raise ValueError(f"the matrix's tensors must be on mx's device, {mx.device}")
            if row_ptr is None and fmt in ("csr", HSS_FMT_CSR):
                row_ptr = torch.zeros(int(m) + 1, dtype=torch.int32, device=mx.device)
            self.flags |= HSS_MX4 | (HSS_MX4_T if mx_t else 0)
        elif mx_t:
            raise ValueError("mx_t without mx")
        self.m, self.n = int(m), int(n)
        self.dtype = dtype
        self.U, self.Vt = U, Vt
        if self.hier_r is not None:
            self.flags |= HSS_HIER2
            self.r = sum(self.hier_r)
            ru = self.hier_r[0] + self.hier_r[1]
            if self.r > 0:
                assert U.shape == (self.m, ru) and Vt.shape == (self.r, self.n - self.n // 2)
        else:
            self.r = 0 if U is None else int(U.shape[1])
            if self.r > 0:
                assert U.shape == (self.m, self.r) and Vt.shape == (self.r, self.n)
        if self.r > 0:
            assert U.dtype == dtype and Vt.dtype == dtype and U.is_contiguous() and Vt.is_contiguous()
        self.row_ptr, self.col_idx, self.values = row_ptr, col_idx, values
        self.nm_values, self.nm_meta = nm_values, nm_meta
        held = (U, Vt, row_ptr, col_idx, values, nm_values, nm_meta, dq_codes, dq_levels,
                None if mx is None else mx.codes)
        on = {t.get_device() for t in held if t is not None}
        self.index = on.pop() if len(on) == 1 else None  # the GPU that holds all of it
        self.nnz = int(nnz if nnz is not None else (values.numel() if values is not None else 0))
        # what the kernels would read out of range, or as other numbers than they are
        if self.fmt == HSS_FMT_CSR:
            self._need("row_ptr", row_ptr, (torch.int32,), self.m + 1)
            if self.nnz > 0:
                self._need("col_idx", col_idx, (torch.int32, torch.int16), self.nnz)
                self._need("values", values, (dtype,), self.nnz)
        else:
            self._need("nm_values", nm_values, (dtype,), self.m * (self.n // 2))
            self._need("nm_meta", nm_meta, (torch.int32,), self.m * ((self.n + 31) // 32))
        self._ws, self._ws_sizes = {}, {}
        s = HssMatrixStruct()
        s.fmt, s.dtype = self.fmt, _DT[dtype]
        s.m, s.n, s.r, s.flags = self.m, self.n, self.r, self.flags
        s.nnz = self.nnz
        s.row_ptr, s.col_idx, s.values = _ptr(row_ptr), _ptr(col_idx), _ptr(values)
        s.nm_values, s.nm_meta = _ptr(nm_values), _ptr(nm_meta)
        s.U, s.Vt = (_ptr(U), _ptr(Vt)) if self.r > 0 else (None, None)
        s.dq_codes, s.dq_levels = _ptr(dq_codes), _ptr(dq_levels)
        if self.hier_r is not None:
            s.hier_r = (ctypes.c_int32 * 4)(*self.hier_r)
        if mx is not None:
            s.dq_codes, s.dq_levels = _ptr(mx.codes), _ptr(mx.scales)
        self.struct = s
        self._ref = ctypes.byref(s)

    @staticmethod
    def _need(name, t, dtypes, count):
        if t is None or t.dtype not in dtypes or t.numel() < count or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor of {count} {' or '.join(str(d) for d in dtypes)}")

    @classmethod
    def from_split(cls, sp: SplitResult, U=None, V=None, Vt=None, dtype=None, mx=None):
        if V is not None:
            Vt = V.t().contiguous()
        if dtype is None:
            dtype = (sp.values if sp.values is not None else sp.nm_values).dtype
        if sp.fmt == HSS_FMT_CSR:
            return cls("csr", sp.m, sp.n, dtype, U=U, Vt=Vt, row_ptr=sp.row_ptr,
                       col_idx=sp.col_idx, values=sp.values, nnz=sp.k, mx=mx)
        if mx is not None:
            raise ValueError("a microscaled dense part goes with a CSR S")
        return cls("2:4", sp.m, sp.n, dtype, U=U, Vt=Vt, nm_values=sp.nm_values, nm_meta=sp.nm_meta)

    def with_col16(self) -> "HSSMatrix":
        """The same CSR matrix with 16-bit columns (converted on the device)."""
        if self.fmt != HSS_FMT_CSR:
            raise ValueError("16-bit columns are a CSR option")
        c16 = hss_csr_cols_to_u16(self.col_idx, self.n) if self.nnz > 0 else None
        return HSSMatrix("csr", self.m, self.n, self.dtype, U=self.U, Vt=self.Vt, row_ptr=self.row_ptr,
                         col_idx=c16 if c16 is not None else torch.zeros(0, dtype=torch.int16,
                                                                           device=self.row_ptr.device),
                         values=self.values, nnz=self.nnz, dq_codes=self.dq_codes, dq_levels=self.dq_levels,
                         hier_r=self.hier_r, mx=self.mx, mx_t=self.mx_t)

    def workspace(self, b: int, device=None) -> torch.Tensor:
        """Initialised apply workspace for batch b on the current stream.

        Cached per (device, stream, size): the decode kernel keeps state in
        its workspace from call to call, so calls that may overlap in time --
        those on different streams -- must not share one.  Calls on one
        stream are ordered and share it safely."""
        size = self._ws_sizes.get(b)
        if size is None:
            size = self._ws_sizes[b] = hss_apply_workspace_size(self, b)
        if device is None:
            held = [t for t in (self.U, self.row_ptr, self.values, self.nm_values, self.dq_codes) if t is not None]
            device = held[0].device
        dev = torch.device(device)
        key = (str(dev), _stream(dev), size)
        if key not in self._ws:
            if torch.cuda.is_current_stream_capturing():
                # its init kernel would be captured too and reset the state on
                # every replay, so that replays could take each other's T words
                raise RuntimeError("create the workspace before graph capture and pass it as ws=")
            self._ws[key] = apply_workspace(size, dev)
        return self._ws[key]


def hss_apply_workspace_init(ws: torch.Tensor) -> torch.Tensor:
    """Put an apply workspace in its initial state (a kernel on the current
    stream); call once before its first apply."""
    with _on(ws):
        check(lib.hss_apply_workspace_init(_ptr(ws), ws.numel(), _stream(ws.device)), "hss_apply_workspace_init")
    return ws


def apply_workspace(size: int, device) -> torch.Tensor:
    """A new apply workspace of `size` bytes on `device`, initialised on the
    current stream.  Calls that share it must be ordered (one stream, or
    events between streams)."""
    ws = torch.empty(max(int(size), 1), dtype=torch.uint8, device=device)
    return hss_apply_workspace_init(ws)


def hss_apply_workspace_size(A: HSSMatrix, b: int) -> int:
    out = ctypes.c_size_t(0)
    check(lib.hss_apply_workspace_size(ctypes.byref(A.struct), int(b), ctypes.byref(out)),
          "hss_apply_workspace_size")
    return int(out.value)


def _check_x(A: HSSMatrix, X: torch.Tensor, index: int) -> int:
    shape = X.shape
    if len(shape) != 2 or shape[1] != A.n or not X.is_contiguous() or X.dtype != A.dtype:
        raise ValueError("X must be a contiguous b x n tensor of the matrix dtype")
    if A.index != index:
        raise ValueError(f"the matrix must be on X's device, {X.device}, with all its tensors")
    return shape[0]


def _check_y(A: HSSMatrix, Y: torch.Tensor, b: int, index: int) -> None:
    if Y.shape != (b, A.m) or Y.dtype != A.dtype or not Y.is_contiguous() or Y.get_device() != index:
        raise ValueError("Y must be a contiguous b x m tensor of the matrix dtype, on X's device")


def _check_ws(ws: torch.Tensor, index: int) -> None:
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the device of the call's other tensors")


def hss_apply(A: HSSMatrix, X: torch.Tensor, Y: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y (b x m) = X (b x n) (S + U V^T)^T on the current stream."""
    index = X.get_device()
    if index < 0:
        _index(X)  # refuses it
    if index != _current_device():
        with torch.cuda.device(index):
            return hss_apply(A, X, Y, ws)
    # the checks of _check_x, _check_y and _check_ws, written out: two calls less in a decode step
    shape, dtype = X.shape, A.dtype
    if len(shape) != 2 or shape[1] != A.n or X.dtype != dtype or A.index != index or not X.is_contiguous():
        _check_x(A, X, index)
    b = shape[0]
    if Y is None:
        Y = torch.empty((b, A.m), dtype=dtype, device=X.device)
    elif Y.shape != (b, A.m) or Y.dtype != dtype or Y.get_device() != index or not Y.is_contiguous():
        _check_y(A, Y, b, index)
    if ws is None:
        ws = A.workspace(b, X.device)
    elif ws.get_device() != index or not ws.is_contiguous():
        _check_ws(ws, index)
    code = lib.hss_apply(A._ref, b, X.data_ptr(), Y.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(index))
    if code:
        check(code, "hss_apply")
    return Y


def hss_apply_noalloc(A: HSSMatrix, X: torch.Tensor, Y: torch.Tensor) -> torch.Tensor:
    """Y (b x m, preallocated) = X (b x n) (S + U V^T)^T on the current stream,
    with the library's own per-GPU scratch instead of a workspace: the call
    allocates nothing.  Calls that overlap in time on one GPU race."""
    index = _index(X)
    if index != _current_device():
        with torch.cuda.device(index):
            return hss_apply_noalloc(A, X, Y)
    b = _check_x(A, X, index)
    _check_y(A, Y, b, index)
    code = lib.hss_apply_noalloc(A._ref, b, X.data_ptr(), Y.data_ptr(), _raw_stream(index))
    if code:
        check(code, "hss_apply_noalloc")
    return Y


def _group_structs(As):
    arr = (ctypes.POINTER(HssMatrixStruct) * len(As))(*[ctypes.pointer(A.struct) for A in As])
    return arr


def hss_apply_group_workspace_size(As, b: int) -> int:
    out = ctypes.c_size_t(0)
    check(lib.hss_apply_group_workspace_size(_group_structs(As), len(As), int(b), ctypes.byref(out)),
          "hss_apply_group_workspace_size")
    return int(out.value)


def hss_apply_group(As, X: torch.Tensor, Ys=None, ws: Optional[torch.Tensor] = None):
    """Y_g = X (S_g + U_g V_g^T)^T for every matrix of As (same n, dtype and
    format), in one launch per decode pass; returns the list of Y_g."""
    index = _index(X)
    if index != _current_device():
        with torch.cuda.device(index):
            return hss_apply_group(As, X, Ys, ws)
    As, b = list(As), 0
    for A in As:
        b = _check_x(A, X, index)
    if Ys is None:
        Ys = [torch.empty((b, A.m), dtype=A.dtype, device=X.device) for A in As]
    elif len(Ys) != len(As):
        raise ValueError(f"{len(As)} matrices, {len(Ys)} outputs")
    else:
        for A, Y in zip(As, Ys):
            _check_y(A, Y, b, index)
    if ws is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("create the workspace before graph capture and pass it as ws=")
        ws = apply_workspace(hss_apply_group_workspace_size(As, b), X.device)
    else:
        _check_ws(ws, index)
    yp = (ctypes.c_void_p * len(As))(*[_ptr(Y) for Y in Ys])
    check(lib.hss_apply_group(_group_structs(As), len(As), b, _ptr(X), yp, _ptr(ws), ws.numel(),
                              _raw_stream(index)), "hss_apply_group")
    return Ys


def hss_csr_cols_to_u16(col_idx: torch.Tensor, n: int) -> torch.Tensor:
    """16-bit copy of int32 CSR columns (n <= 65536), as a torch.int16 tensor
    holding the uint16 bit patterns."""
    dev = _dev(col_idx)
    if col_idx.dtype != torch.int32 or not col_idx.is_contiguous():
        raise ValueError("col_idx must be a contiguous int32 tensor")
    out = torch.empty(col_idx.numel(), dtype=torch.int16, device=dev)
    with _on(col_idx):
        check(lib.hss_csr_cols_to_u16(_ptr(col_idx), col_idx.numel(), int(n), _ptr(out), _stream(dev)),
              "hss_csr_cols_to_u16")
    return out


# ---------------------------------------------------------------------------
# Hierarchical variant
# ---------------------------------------------------------------------------

def hss_rcm_order(row_ptr, col_idx, n: int):
    """Reverse Cuthill-McKee order of a square CSR pattern (host arrays, or
    tensors copied to the host): numpy int32 perm, perm[i] = original index
    at position i."""
    import numpy as np
    rp = np.ascontiguousarray(row_ptr.cpu().numpy() if isinstance(row_ptr, torch.Tensor) else row_ptr, dtype=np.int32)
    ci = np.ascontiguousarray(col_idx.cpu().numpy() if isinstance(col_idx, torch.Tensor) else col_idx, dtype=np.int32)
    perm = np.zeros(int(n), dtype=np.int32)
    check(lib.hss_rcm_order(int(n), rp.ctypes.data, ci.ctypes.data if ci.size else None, perm.ctypes.data),
          "hss_rcm_order")
    return perm


def hss_concentration(W: torch.Tensor, perm: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Device float64 tensor [rho, diagonal-block |W| sum, total |W| sum] of W
    (rows and columns in the order perm, a device int32 permutation)."""
    dev = _dev(W)
    if W.dim() != 2 or not W.is_contiguous() or W.dtype not in _DT:
        raise ValueError("W must be a contiguous 2-D fp32 or bf16 tensor")
    m, n = W.shape
    size = ctypes.c_size_t(0)
    check(lib.hss_concentration_workspace_size(m, n, ctypes.byref(size)), "hss_concentration_workspace_size")
    ws = torch.empty(size.value, dtype=torch.uint8, device=dev)
    out = torch.empty(3, dtype=torch.float64, device=dev)
    if perm is not None and (perm.dtype != torch.int32 or perm.numel() != n or not perm.is_contiguous()):
        raise ValueError("perm must be a contiguous int32 tensor of n entries")
    with _on(W):
        check(lib.hss_concentration(_DT[W.dtype], m, n, _ptr(W), _ptr(perm), _ptr(out), _ptr(ws), ws.numel(),
                                    _stream(dev)), "hss_concentration")
    return out


def hss_hier_pack(U, Vt, m: int, n: int, perm: Optional[torch.Tensor] = None):
    """Flat factors (U_cat m x R, Vt_cat R x n) of the 2 x 2 block low-rank
    term with blocks U[b] Vt[b], b in the order 00, 01, 10, 11, on the matrix
    permuted by perm (device int32 or None)."""
    dtype = next(u.dtype for u in U if u is not None)
    dev = next(u.device for u in U if u is not None)
    r = [0 if u is None else int(u.shape[1]) for u in U]
    R = sum(r)
    Ucat = torch.empty((m, R), dtype=dtype, device=dev)
    Vtcat = torch.empty((R, n), dtype=dtype, device=dev)
    rows, cols = (m // 2, m - m // 2), (n // 2, n - n // 2)
    for b, (u, v) in enumerate(zip(U, Vt)):
        if u is None:
            continue
        if not u.is_contiguous() or not v.is_contiguous() or u.dtype != dtype or v.dtype != dtype:
            raise ValueError("blocks must be contiguous tensors of one dtype")
        if tuple(u.shape) != (rows[b >> 1], r[b]) or tuple(v.shape) != (r[b], cols[b & 1]):
            raise ValueError(f"block {b}: U {tuple(u.shape)} / Vt {tuple(v.shape)} do not fit a {m} x {n} matrix")
    r_arr = (ctypes.c_int32 * 4)(*r)
    u_arr = (ctypes.c_void_p * 4)(*[_ptr(u) for u in U])
    v_arr = (ctypes.c_void_p * 4)(*[_ptr(v) for v in Vt])
    with _on(Ucat):
        check(lib.hss_hier_pack(_DT[dtype], int(m), int(n), r_arr, u_arr, v_arr, _ptr(perm), _ptr(Ucat), _ptr(Vtcat),
                                _stream(dev)), "hss_hier_pack")
    return Ucat, Vtcat


def hss_hier_pack_compact(U, Vt, m: int, n: int):
    """Compact factors (U_c m x ru, Vt_c R x (n - n // 2)) of an HSS_HIER2
    matrix from its blocks U[b] Vt[b], b in the order 00, 01, 10, 11 (None
    for a rank-0 block), in the blocks' own order; with hier_r = the block
    ranks they make HSSMatrix(..., hier_r=...)."""
    dtype = next(u.dtype for u in U if u is not None)
    dev = next(u.device for u in U if u is not None)
    r = [0 if u is None else int(u.shape[1]) for u in U]
    R, ru = sum(r), r[0] + r[1]
    rows, cols = (m // 2, m - m // 2), (n // 2, n - n // 2)
    for b, (u, v) in enumerate(zip(U, Vt)):
        if u is None:
            continue
        if not u.is_contiguous() or not v.is_contiguous() or u.dtype != dtype or v.dtype != dtype:
            raise ValueError("blocks must be contiguous tensors of one dtype")
        if tuple(u.shape) != (rows[b >> 1], r[b]) or tuple(v.shape) != (r[b], cols[b & 1]):
            raise ValueError(f"block {b}: U {tuple(u.shape)} / Vt {tuple(v.shape)} do not fit a {m} x {n} matrix")
    Uc = torch.empty((m, ru), dtype=dtype, device=dev)
    Vtc = torch.empty((R, n - n // 2), dtype=dtype, device=dev)
    r_arr = (ctypes.c_int32 * 4)(*r)
    u_arr = (ctypes.c_void_p * 4)(*[_ptr(u) for u in U])
    v_arr = (ctypes.c_void_p * 4)(*[_ptr(v) for v in Vt])
    with _on(Uc):
        check(lib.hss_hier_pack_compact(_DT[dtype], int(m), int(n), r_arr, u_arr, v_arr, _ptr(Uc), _ptr(Vtc),
                                        _stream(dev)), "hss_hier_pack_compact")
    return Uc, Vtc


def hss_csr_permute(row_ptr, col_idx, perm, n: int):
    """S' = P S P^T (S'[i][j] = S[perm[i]][perm[j]]) of a square CSR pattern,
    on the host: (row_ptr_p, col_idx_p, from), entry q of S' being entry
    from[q] of S (hss_gather_values moves the values)."""
    import numpy as np
    rp = np.ascontiguousarray(row_ptr.cpu().numpy() if isinstance(row_ptr, torch.Tensor) else row_ptr, dtype=np.int32)
    ci = np.ascontiguousarray(col_idx.cpu().numpy() if isinstance(col_idx, torch.Tensor) else col_idx, dtype=np.int32)
    pm = np.ascontiguousarray(perm.cpu().numpy() if isinstance(perm, torch.Tensor) else perm, dtype=np.int32)
    nnz = int(rp[n])
    rpp = np.zeros(int(n) + 1, dtype=np.int32)
    cip = np.zeros(max(nnz, 1), dtype=np.int32)
    frm = np.zeros(max(nnz, 1), dtype=np.int32)
    check(lib.hss_csr_permute(int(n), rp.ctypes.data, ci.ctypes.data if nnz else None, pm.ctypes.data,
                              rpp.ctypes.data, cip.ctypes.data, frm.ctypes.data), "hss_csr_permute")
    return rpp, cip[:nnz], frm[:nnz]



# ---------------------------------------------------------------------------
# Backward pass
# ---------------------------------------------------------------------------

def hss_grad(A: HSSMatrix, X: torch.Tensor, G: torch.Tensor, dS=True, dU=True, dVt=True,
             ws: Optional[torch.Tensor] = None) -> dict:
    """Parameter gradients of a bf16 layer (CSR or 2:4) for the upstream
    gradient G (b x m): fp32 dS (S's stored values, storage order: nnz for
    CSR, m x n/2 laid out as nm_values for 2:4), dU (m x r) and dVt (r x n,
    the gradient of the stored V^T).  Pass False to skip one."""
    dev = _dev(X)
    if X.dim() != 2 or X.shape[1] != A.n or not X.is_contiguous() or X.dtype != A.dtype:
        raise ValueError("X must be a contiguous b x n tensor of the matrix dtype")
    b = X.shape[0]
    index = X.get_device()
    if G.shape != (b, A.m) or not G.is_contiguous() or G.dtype != A.dtype or G.get_device() != index:
        raise ValueError("G must be a contiguous b x m tensor of the matrix dtype, on X's device")
    if A.index != index:
        raise ValueError(f"the matrix must be on X's device, {X.device}, with all its tensors")
    out = {}
    if dS:
        stored = A.m * (A.n // 2) if A.fmt == HSS_FMT_2OF4 else A.nnz
        out["dS"] = torch.empty(stored, dtype=torch.float32, device=dev)
    if dU:
        out["dU"] = torch.empty((A.m, A.r), dtype=torch.float32, device=dev)
    if dVt:
        out["dVt"] = torch.empty((A.r, A.n), dtype=torch.float32, device=dev)
    if ws is None:
        size = ctypes.c_size_t(0)
        check(lib.hss_grad_workspace_size(ctypes.byref(A.struct), b, ctypes.byref(size)), "hss_grad_workspace_size")
        ws = torch.empty(size.value, dtype=torch.uint8, device=dev)
    else:
        _check_ws(ws, index)
    with _on(X):
        check(lib.hss_grad(ctypes.byref(A.struct), b, _ptr(X), _ptr(G), _ptr(out.get("dS")), _ptr(out.get("dU")),
                           _ptr(out.get("dVt")), _ptr(ws), ws.numel(), _stream(dev)), "hss_grad")
    return out


def hss_csr_transpose(row_ptr, col_idx, m: int, n: int):
    """S^T's CSR pattern (host int32 row_ptr_t, col_idx_t) and perm (entry q of
    S^T is entry perm[q] of S), computed on the host."""
    import numpy as np
    rp = np.ascontiguousarray(row_ptr.cpu().numpy() if isinstance(row_ptr, torch.Tensor) else row_ptr, dtype=np.int32)
    ci = np.ascontiguousarray(col_idx.cpu().numpy() if isinstance(col_idx, torch.Tensor) else col_idx, dtype=np.int32)
    nnz = int(rp[m])
    rpt = np.zeros(int(n) + 1, dtype=np.int32)
    cit = np.zeros(max(nnz, 1), dtype=np.int32)
    perm = np.zeros(max(nnz, 1), dtype=np.int32)
    check(lib.hss_csr_transpose(int(m), int(n), rp.ctypes.data, ci.ctypes.data if nnz else None, rpt.ctypes.data,
                                cit.ctypes.data, perm.ctypes.data), "hss_csr_transpose")
    return rpt, cit[:nnz], perm[:nnz]


def hss_gather_values(values: torch.Tensor, perm: torch.Tensor) -> torch.Tensor:
    """values[perm] on the device (bits copied); perm int32, within values."""
    if values.dtype not in _DT or not values.is_contiguous():
        raise ValueError("values must be a contiguous fp32 or bf16 tensor")
    if perm.dtype != torch.int32 or not perm.is_contiguous() or perm.get_device() != values.get_device():
        raise ValueError("perm must be a contiguous int32 tensor on the device of values")
    out = torch.empty(perm.numel(), dtype=values.dtype, device=values.device)
    with _on(values):
        check(lib.hss_gather_values(_DT[values.dtype], perm.numel(), _ptr(values), _ptr(perm), _ptr(out),
                                    _stream(values.device)), "hss_gather_values")
    return out


def hss_transpose(t: torch.Tensor) -> torch.Tensor:
    """A contiguous 2-D fp32 / bf16 device tensor transposed by the library."""
    if t.dim() != 2 or not t.is_contiguous() or t.dtype not in _DT:
        raise ValueError("t must be a contiguous 2-D fp32 or bf16 tensor")
    rows, cols = t.shape
    out = torch.empty((cols, rows), dtype=t.dtype, device=t.device)
    with _on(t):
        check(lib.hss_transpose(_DT[t.dtype], rows, cols, _ptr(t), _ptr(out), _stream(t.device)), "hss_transpose")
    return out


def hss_nm24_to_csr(A: HSSMatrix):
    """The stored positions of a 2:4 matrix as a device CSR pattern (row_ptr,
    col_idx) in storage order: its values array is nm_values flattened."""
    dev = A.nm_meta.device
    rp = torch.empty(A.m + 1, dtype=torch.int32, device=dev)
    ci = torch.empty(A.m * (A.n // 2), dtype=torch.int32, device=dev)
    with _on(A.nm_meta):
        check(lib.hss_nm24_to_csr(A.m, A.n, _ptr(A.nm_meta), _ptr(rp), _ptr(ci), _stream(dev)), "hss_nm24_to_csr")
    return rp, ci


def _rewrite_transposed(A: HSSMatrix, out: HSSMatrix) -> HSSMatrix:
    """A's values and factors into the transposed layer `out`: no host work, no allocation."""
    nnz = A.m * (A.n // 2) if A.fmt == HSS_FMT_2OF4 else A.nnz
    perm = getattr(out, "perm_from_s", None)
    if perm is None or (out.m, out.n, out.r, out.dtype, out.nnz) != (A.n, A.m, A.r, A.dtype, nnz) or \
            out.mx is not A.mx or (A.mx is not None and out.mx_t == A.mx_t) or out.index != A.index:
        raise ValueError("out must be a transposed layer that hss_transposed_layer made of a layer like A")
    held = out.row_ptr
    with _on(held):
        stream = _stream(held.device)
        if nnz:
            values = A.nm_values if A.fmt == HSS_FMT_2OF4 else A.values
            check(lib.hss_gather_values(_DT[A.dtype], nnz, _ptr(values), _ptr(perm), _ptr(out.values), stream),
                  "hss_gather_values")
        if A.r > 0:
            check(lib.hss_transpose(_DT[A.dtype], A.r, A.n, _ptr(A.Vt), _ptr(out.U), stream), "hss_transpose")
            check(lib.hss_transpose(_DT[A.dtype], A.m, A.r, _ptr(A.U), _ptr(out.Vt), stream), "hss_transpose")
    return out


def hss_transposed_layer(A: HSSMatrix, out: Optional[HSSMatrix] = None) -> HSSMatrix:
    """A^T = S^T + V U^T as an HSSMatrix (n x m, CSR): S^T's pattern from the
    host transpose (of the 2:4 positions for a 2:4 layer), its values
    gathered on the device, U' = V and V'^T = U^T from the stored factors; a
    microscaled dense part is shared, read transposed.  hss_apply(A^T, G) is the input gradient G A.

    S's values, U and V are copied: after they change (an optimizer's step),
    out = the layer this call returned before writes them again from A's, in
    place and on the device (S's pattern must be the same)."""
    if A.flags & (HSS_DQ4 | HSS_HIER2):
        raise ValueError("the transposed layer is built for CSR and 2:4 layers with flat factors")
    if out is not None:
        return _rewrite_transposed(A, out)
    mx = dict(mx=A.mx, mx_t=not A.mx_t) if A.mx is not None else {}
    if A.fmt == HSS_FMT_2OF4:
        dev = A.nm_meta.device
        row_ptr, cols = hss_nm24_to_csr(A)
        values, nnz = A.nm_values.reshape(-1), A.m * (A.n // 2)
    else:
        dev = A.row_ptr.device
        row_ptr, values, nnz = A.row_ptr, A.values, A.nnz
        cols = A.col_idx.to(torch.int32) if A.flags & HSS_COL16 else A.col_idx
        if A.flags & HSS_COL16:
            cols = cols & 0xFFFF
    rpt, cit, perm = hss_csr_transpose(row_ptr, cols if nnz else torch.zeros(0, dtype=torch.int32), A.m, A.n)
    perm_d = torch.from_numpy(perm).to(dev)
    vals = hss_gather_values(values, perm_d) if nnz else None
    U2 = hss_transpose(A.Vt) if A.r > 0 else None
    Vt2 = hss_transpose(A.U) if A.r > 0 else None
    At = HSSMatrix("csr", A.n, A.m, A.dtype, U=U2, Vt=Vt2, row_ptr=torch.from_numpy(rpt).to(dev),
                   col_idx=torch.from_numpy(cit).to(dev) if nnz else None, values=vals, nnz=nnz, **mx)
    At.perm_from_s = perm_d
    return At


def hss_grad_ckpt_workspace_size(A: HSSMatrix, b: int) -> int:
    out = ctypes.c_size_t(0)
    check(lib.hss_grad_ckpt_workspace_size(ctypes.byref(A.struct), int(b), ctypes.byref(out)),
          "hss_grad_ckpt_workspace_size")
    return int(out.value)


def grad_ckpt_workspace(A: HSSMatrix, b: int, device) -> torch.Tensor:
    """A workspace of hss_grad_ckpt for batch b.  It keeps no state between
    calls; calls that share it must be ordered (one stream, or events)."""
    return torch.empty(hss_grad_ckpt_workspace_size(A, b), dtype=torch.uint8, device=device)


def hss_grad_ckpt(A: HSSMatrix, X: MXTensor, G: torch.Tensor, dS=True, dU=True, dVt=True,
                  out: Optional[dict] = None, ws: Optional[torch.Tensor] = None) -> dict:
    """hss_grad with the layer's input as an 8-bit checkpoint: X is the "int8"
    MXTensor (b x n) that hss_mx_quantize made of it in the forward pass.
    out: tensors to write (a dict with the keys wanted, as returned); then
    dS, dU and dVt are ignored."""
    index, dev = _index(G), G.device
    if index != _current_device():
        with torch.cuda.device(index):
            return hss_grad_ckpt(A, X, G, dS, dU, dVt, out, ws)
    if X.fmt != "int8" or X.cols != A.n or X.index != index:
        raise ValueError("X must be an 'int8' MXTensor, b x n, on G's device")
    if A.index != index:
        raise ValueError(f"the matrix must be on G's device, {dev}, with all its tensors")
    b = X.rows
    if G.shape != (b, A.m) or not G.is_contiguous() or G.dtype != A.dtype:
        raise ValueError("G must be a contiguous b x m tensor of the matrix dtype")
    shapes = {"dS": (A.m * (A.n // 2) if A.fmt == HSS_FMT_2OF4 else A.nnz,), "dU": (A.m, A.r), "dVt": (A.r, A.n)}
    if out is None:
        out = {k: torch.empty(shapes[k], dtype=torch.float32, device=dev)
               for k, wanted in (("dS", dS), ("dU", dU), ("dVt", dVt)) if wanted}
    else:
        for k, t in out.items():
            if k not in shapes or t.shape != shapes[k] or t.dtype != torch.float32 or not t.is_contiguous() or \
                    t.get_device() != index:
                raise ValueError("out must hold contiguous float32 tensors 'dS', 'dU', 'dVt' of the gradients' shapes")
    if ws is None:
        ws = grad_ckpt_workspace(A, b, dev)
    else:
        _check_ws(ws, index)
    check(lib.hss_grad_ckpt(ctypes.byref(A.struct), b, X.codes.data_ptr(), X.scales.data_ptr(), G.data_ptr(),
                            _ptr(out.get("dS")), _ptr(out.get("dU")), _ptr(out.get("dVt")), ws.data_ptr(),
                            ws.numel(), _raw_stream(index)), "hss_grad_ckpt")
    return out


def hss_backward(A: HSSMatrix, X, G: torch.Tensor, At: Optional[HSSMatrix] = None) -> dict:
    """dX (b x n, the layer dtype) = G A through the transposed layer, and
    the fp32 parameter gradients dS, dU, dVt of hss_grad, or of hss_grad_ckpt
    where X is the 8-bit checkpoint of the layer's input.  At: the transposed
    layer, of A's present values (hss_transposed_layer(A, out=At) writes them
    again); without it one is made, with S's pattern transposed on the host."""
    if At is None:
        At = hss_transposed_layer(A)
    out = hss_grad_ckpt(A, X, G) if isinstance(X, MXTensor) else hss_grad(A, X, G)
    out["dX"] = hss_apply(At, G)
    return out
