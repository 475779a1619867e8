"""LLM.int8() matrix multiplication for NVIDIA B200 (sm_100a).

Python face of ``libint8mm`` (C-ABI in ``include/int8mm.h``).  PyTorch is used
for device memory and streams only; every step of the product runs in the
library's CUDA kernels, and there is no CPU fallback.

Method: "LLM.int8(): 8-bit Matrix Multiplication for Transformers at Scale"
(Dettmers et al., 2022), abstract -- vector-wise int8 quantisation plus a
16-bit matmul over the outlier feature dimensions, for the feed-forward and
attention-projection layers of a transformer.

    w  = prepare_weight(W_fp16_KxN, keep_idx)      # once, at load
    ws = Workspace(M, K, N)                         # reusable scratch
    Y  = forward(X_fp16_MxK, w, threshold=6.0, workspace=ws)

The same layers with block-scaled e4m3 codes (fp16 or bf16 tensors), and a
mixture-of-experts layer of them for a few tokens:

    w8 = prepare_weight_fp8(W_KxN)                  # or weight_fp8(codes, scales)
    Y  = forward_fp8(X_MxK, w8, workspace=Fp8Workspace(M, K, N))
    m  = prepare_moe_weight_fp8(router, gate, up, down)
    Y  = forward_moe_fp8(X_TxH, m, top_k, workspace=MoeWorkspace(T, m, top_k))

These e4m3 calls take stream=s as a ``with torch.cuda.stream(s)`` around them
does: s has to wait for whatever wrote the inputs, and what a call allocates
belongs to s.  The memory of what a call is given is kept until s is done.
The int8, 4-bit and codec calls launch on s too, but allocate on the current
stream: with stream=s give them their outputs and workspace, and keep every
tensor until s is done.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _abi
from ._abi import PATH_AUTO, PATH_DECODE, PATH_GEMM, PATH_GEMM_1SM, Int8mmError

__all__ = [
    "PreparedWeight", "Workspace", "prepare_weight", "forward", "device_status", "library",
    "block_quantize", "block_dequantize",
    "Int4Weight", "prepare_weight_int4", "forward_int4", "unpack_int4_codes",
    "GroupedWeight", "prepare_weight_grouped", "forward_grouped",
    "Fp8Weight", "Fp8Workspace", "quantize_fp8", "prepare_weight_fp8", "weight_fp8", "forward_fp8",
    "MoeFp8Weight", "MoeWorkspace", "prepare_moe_weight_fp8", "moe_weight_fp8", "forward_moe_fp8",
    "Int8mmError", "PATH_AUTO", "PATH_GEMM", "PATH_DECODE",
]

_PATHS = {"auto": PATH_AUTO, "gemm": PATH_GEMM, "decode": PATH_DECODE, "gemm1sm": PATH_GEMM_1SM}


def library():
    """The loaded ctypes handle of libint8mm.so (raises if it is missing)."""
    return _abi.load()


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _view(buf: torch.Tensor, ptr: int, count: int, dtype: torch.dtype, shape=None) -> torch.Tensor:
    off = int(ptr) - buf.data_ptr()
    nbytes = count * torch.empty(0, dtype=dtype).element_size()
    t = buf[off: off + nbytes].view(dtype)
    return t.view(*shape) if shape is not None else t


class PreparedWeight:
    """An int8 weight in one device buffer (see ``int8mm_weight`` in the header)."""

    def __init__(self, buf: torch.Tensor, st: _abi.Weight):
        self.buf = buf
        self.struct = st
        self.K, self.N, self.n_keep = st.K, st.N, st.n_keep

    @property
    def wq(self) -> torch.Tensor:           # N x K int8
        return _view(self.buf, self.struct.wq, self.N * self.K, torch.int8, (self.N, self.K))

    @property
    def col_absmax(self) -> torch.Tensor:   # N float32
        return _view(self.buf, self.struct.col_absmax, self.N, torch.float32)

    @property
    def w_keep(self) -> torch.Tensor:       # n_keep x N fp16
        return _view(self.buf, self.struct.w_keep, self.n_keep * self.N, torch.float16, (self.n_keep, self.N))

    @property
    def keep_idx(self) -> torch.Tensor:
        return _view(self.buf, self.struct.keep_idx, self.n_keep, torch.int32)


def prepare_weight(W: torch.Tensor, keep_idx=(), stream=None) -> PreparedWeight:
    """Convert a K x N fp16 CUDA weight to int8 once (at load, per the LLM.int8() abstract)."""
    lib = _abi.load()
    if not (W.is_cuda and W.dtype == torch.float16 and W.dim() == 2 and W.is_contiguous()):
        raise ValueError("W must be a contiguous 2-D float16 CUDA tensor (K x N)")
    K, N = W.shape
    keep = np.unique(np.asarray(keep_idx, dtype=np.int64).ravel()).astype(np.int32)
    nbytes = lib.int8mm_weight_bytes(K, N, int(keep.size))
    if nbytes == 0:
        raise Int8mmError(1, f"int8mm_weight_bytes(K={K}, N={N}, n_keep={keep.size})")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    st = _abi.Weight()
    kp = keep.ctypes.data_as(ctypes.c_void_p) if keep.size else None
    with torch.cuda.device(W.device):
        _abi.check(lib.int8mm_prepare_weight(ctypes.c_void_p(W.data_ptr()), K, N, kp, int(keep.size),
                                             ctypes.c_void_p(buf.data_ptr()), nbytes, ctypes.byref(st),
                                             _stream(stream)), "int8mm_prepare_weight")
    return PreparedWeight(buf, st)


class Workspace:
    """Device scratch of one forward shape; zero-filled at creation."""

    def __init__(self, M: int, K: int, N: int, max_outliers: int | None = None, device=None, G: int | None = None):
        """G: group size of a group-wise forward (None: vector-wise)."""
        lib = _abi.load()
        self.M, self.K, self.N, self.G = M, K, N, G
        self.max_outliers = K if max_outliers is None else int(max_outliers)
        if G is None:
            self.nbytes = lib.int8mm_workspace_bytes(M, K, N, self.max_outliers)
        else:
            self.nbytes = lib.int8mm_grouped_workspace_bytes(M, K, N, int(G), self.max_outliers)
        if self.nbytes == 0:
            raise Int8mmError(1, f"workspace bytes (M={M}, K={K}, N={N}, max_outliers={self.max_outliers}, G={G})")
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")

    def reset(self, stream=None) -> None:
        """Zero the workspace again (needed after a forward reported a device error)."""
        with torch.cuda.device(self.buf.device):
            _abi.check(_abi.load().int8mm_workspace_init(ctypes.c_void_p(self.buf.data_ptr()), self.nbytes,
                                                         _stream(stream)), "int8mm_workspace_init")

    def view(self) -> dict:
        """Torch views of the intermediates the last forward left in the workspace."""
        v = _abi.WorkspaceView()
        lib = _abi.load()
        if self.G is None:
            _abi.check(lib.int8mm_workspace_view_get(ctypes.c_void_p(self.buf.data_ptr()), self.nbytes, self.M,
                                                     self.K, self.N, self.max_outliers, ctypes.byref(v)),
                       "int8mm_workspace_view_get")
        else:
            _abi.check(lib.int8mm_grouped_workspace_view_get(ctypes.c_void_p(self.buf.data_ptr()), self.nbytes, self.M,
                                                             self.K, self.N, int(self.G), self.max_outliers,
                                                             ctypes.byref(v)), "int8mm_grouped_workspace_view_get")
        nr = 1 if self.G is None else self.K // self.G
        b = self.buf
        return {
            "status": _view(b, v.status, 1, torch.int32),
            "n_outliers": _view(b, v.n_outliers, 1, torch.int32),
            "outlier_idx": _view(b, v.outlier_idx, self.K, torch.int32),
            "row_absmax": (_view(b, v.row_absmax, self.M, torch.float32) if self.G is None else
                           _view(b, v.row_absmax, self.M * nr, torch.float32, (self.M, nr))),
            "xq": _view(b, v.xq, self.M * self.K, torch.int8, (self.M, self.K)),
            "xo": _view(b, v.xo, self.M * v.kp, torch.float16, (self.M, v.kp)) if v.kp else None,
            "kp": v.kp,
        }


def forward(X: torch.Tensor, w: PreparedWeight, threshold: float = 6.0, *, max_outliers: int | None = None,
            out: torch.Tensor | None = None, workspace: Workspace | None = None, path: str = "auto",
            acc_out: torch.Tensor | None = None, wait_limit_ns: int = 0, test_flags: int = 0,
            stream=None) -> torch.Tensor:
    """Y = X W by LLM.int8().  X: M x K fp16.  A CPU X goes through
    int8mm_forward_host (copy in, product, copy back in row bands that overlap
    the product) and a CPU Y (``out``, pinned if given, else a new pinned
    tensor) is returned once it is complete; a CUDA X stays on its device."""
    lib = _abi.load()
    on_host = not X.is_cuda
    dev = w.buf.device
    if X.dtype != torch.float16 or X.dim() != 2 or X.shape[1] != w.K:
        raise ValueError(f"X must be float16 of shape (M, {w.K})")
    if not X.is_contiguous():
        raise ValueError("X must be contiguous")
    M = X.shape[0]
    if on_host:
        if acc_out is not None or path != "auto" or wait_limit_ns or test_flags:
            raise ValueError("a host X takes the default path and options")
        if workspace is None:
            workspace = Workspace(M, w.K, w.N, max_outliers, device=dev)
        if (workspace.M, workspace.K, workspace.N) != (M, w.K, w.N):
            raise ValueError("workspace was made for another shape")
        host = out if out is not None else torch.empty(M, w.N, dtype=torch.float16, pin_memory=True)
        if host.is_cuda or host.shape != (M, w.N) or host.dtype != torch.float16 or not host.is_contiguous():
            raise ValueError("out must be a contiguous CPU float16 tensor of shape (M, N) for a host X")
        Xd = torch.empty(M, w.K, dtype=torch.float16, device=dev)
        Yd = torch.empty(M, w.N, dtype=torch.float16, device=dev)
        with torch.cuda.device(dev):
            st = stream or torch.cuda.current_stream()
            _abi.check(lib.int8mm_forward_host(ctypes.c_void_p(X.data_ptr()), M, ctypes.byref(w.struct),
                                               float(threshold), workspace.max_outliers,
                                               ctypes.c_void_p(host.data_ptr()), ctypes.c_void_p(Xd.data_ptr()),
                                               ctypes.c_void_p(Yd.data_ptr()),
                                               ctypes.c_void_p(workspace.buf.data_ptr()), workspace.nbytes,
                                               _stream(stream)), "int8mm_forward_host")
            st.synchronize()
        return host
    Xd = X
    if workspace is None:
        workspace = Workspace(M, w.K, w.N, max_outliers, device=dev)
    if (workspace.M, workspace.K, workspace.N) != (M, w.K, w.N):
        raise ValueError("workspace was made for another shape")
    Y = out if out is not None else torch.empty(M, w.N, dtype=torch.float16, device=dev)
    opts = _abi.ForwardOpts(_PATHS[path], ctypes.c_void_p(acc_out.data_ptr()) if acc_out is not None else None,
                            int(wait_limit_ns), None, None, int(test_flags))
    with torch.cuda.device(dev):
        _abi.check(lib.int8mm_forward_ex(ctypes.c_void_p(Xd.data_ptr()), M, ctypes.byref(w.struct), float(threshold),
                                         workspace.max_outliers, ctypes.c_void_p(Y.data_ptr()),
                                         ctypes.c_void_p(workspace.buf.data_ptr()), workspace.nbytes,
                                         ctypes.byref(opts), _stream(stream)), "int8mm_forward")
    return Y


def device_status(workspace: Workspace, stream=None) -> tuple[int, int]:
    """(status code, detected outlier count) of the last forward; syncs the stream."""
    n = ctypes.c_int32(0)
    with torch.cuda.device(workspace.buf.device):
        st = _abi.load().int8mm_get_device_status(ctypes.c_void_p(workspace.buf.data_ptr()), _stream(stream),
                                                  ctypes.byref(n))
    return int(st), int(n.value)


# ---------------------------------------------------------------------------- block-wise 8-bit codec

def block_quantize(x: torch.Tensor, B: int, q: torch.Tensor | None = None, absmax: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Block-wise linear 8-bit codes of a float32 CUDA vector: block b covers
    [b*B, min(n, (b+1)*B)) and is normalised by its own absolute maximum
    (axolotl "llama3-model-quantization", "8-Bit Optimizers" paragraphs).
    Returns (codes int8 of n, absmax float32 of ceil(n/B))."""
    if not (x.is_cuda and x.dtype == torch.float32 and x.is_contiguous()):
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    n = x.numel()
    nb = (n + B - 1) // B
    q = torch.empty(n, dtype=torch.int8, device=x.device) if q is None else q
    absmax = torch.empty(nb, dtype=torch.float32, device=x.device) if absmax is None else absmax
    with torch.cuda.device(x.device):
        _abi.check(_abi.load().int8mm_block_quantize(ctypes.c_void_p(x.data_ptr()), n, int(B),
                                                     ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(absmax.data_ptr()),
                                                     _stream(stream)), "int8mm_block_quantize")
    return q, absmax


def block_dequantize(q: torch.Tensor, absmax: torch.Tensor, B: int, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """float32 values (q * absmax[block]) / 127 of block-wise codes."""
    if not (q.is_cuda and q.dtype == torch.int8 and q.is_contiguous()):
        raise ValueError("q must be a contiguous int8 CUDA tensor")
    n = q.numel()
    out = torch.empty(n, dtype=torch.float32, device=q.device) if out is None else out
    with torch.cuda.device(q.device):
        _abi.check(_abi.load().int8mm_block_dequantize(ctypes.c_void_p(q.data_ptr()),
                                                       ctypes.c_void_p(absmax.data_ptr()), n, int(B),
                                                       ctypes.c_void_p(out.data_ptr()), _stream(stream)),
                   "int8mm_block_dequantize")
    return out


# ---------------------------------------------------------------------------- 4-bit weight-only decode product

class Int4Weight:
    """A 4-bit weight in one device buffer (see ``int8mm_int4_weight``)."""

    def __init__(self, buf: torch.Tensor, st: _abi.Int4Weight):
        self.buf = buf
        self.struct = st
        self.K, self.N, self.G = st.K, st.N, st.G

    @property
    def codes(self) -> torch.Tensor:        # N x K/2 packed nibbles
        return _view(self.buf, self.struct.codes, self.N * self.K // 2, torch.uint8, (self.N, self.K // 2))

    @property
    def absmax(self) -> torch.Tensor:       # N x K/G float32
        return _view(self.buf, self.struct.absmax, self.N * (self.K // self.G), torch.float32,
                      (self.N, self.K // self.G))


def prepare_weight_int4(W: torch.Tensor, G: int, stream=None) -> Int4Weight:
    """Convert a K x N fp16 CUDA weight to 4-bit codes with one constant per
    output column and group of G consecutive k (once, at load)."""
    lib = _abi.load()
    if not (W.is_cuda and W.dtype == torch.float16 and W.dim() == 2 and W.is_contiguous()):
        raise ValueError("W must be a contiguous 2-D float16 CUDA tensor (K x N)")
    K, N = W.shape
    nbytes = lib.int8mm_int4_weight_bytes(K, N, int(G))
    if nbytes == 0:
        raise Int8mmError(1, f"int8mm_int4_weight_bytes(K={K}, N={N}, G={G})")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    st = _abi.Int4Weight()
    with torch.cuda.device(W.device):
        _abi.check(lib.int8mm_prepare_weight_int4(ctypes.c_void_p(W.data_ptr()), K, N, int(G),
                                                  ctypes.c_void_p(buf.data_ptr()), nbytes, ctypes.byref(st),
                                                  _stream(stream)), "int8mm_prepare_weight_int4")
    return Int4Weight(buf, st)


def forward_int4(X: torch.Tensor, w: Int4Weight, out: torch.Tensor | None = None,
                 status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X W' with the 4-bit weight (X: M x K fp16 on the weight's device,
    M <= 16).  ``status`` (int32 CUDA tensor of one zero word) receives
    device-side errors; a fresh one is used when it is None."""
    lib = _abi.load()
    if X.dtype != torch.float16 or X.dim() != 2 or X.shape[1] != w.K or not X.is_cuda or not X.is_contiguous():
        raise ValueError(f"X must be a contiguous float16 CUDA tensor of shape (M, {w.K})")
    M = X.shape[0]
    Y = out if out is not None else torch.empty(M, w.N, dtype=torch.float16, device=X.device)
    status = status if status is not None else torch.zeros(1, dtype=torch.int32, device=X.device)
    with torch.cuda.device(X.device):
        _abi.check(lib.int8mm_forward_int4(ctypes.c_void_p(X.data_ptr()), M, ctypes.byref(w.struct),
                                           ctypes.c_void_p(Y.data_ptr()), ctypes.c_void_p(status.data_ptr()),
                                           _stream(stream)), "int8mm_forward_int4")
    return Y


def unpack_int4_codes(packed: np.ndarray) -> np.ndarray:
    """Codes q (N x K int8) from the packed layout (N x K/2 uint8) that
    ``int8mm_int4_weight`` documents; a layout helper, no arithmetic."""
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    N, half = packed.shape
    words = packed.view("<u4").reshape(N, half // 4)
    q = np.empty((N, half * 2), dtype=np.int8)
    for i in range(8):
        shift = (i & 1) * 16 + (i >> 1) * 4
        q[:, i::8] = (((words >> shift) & 0xF).astype(np.int16) - 8).astype(np.int8)
    return q


# ---------------------------------------------------------------------------- group-wise variant

class GroupedWeight:
    """A group-wise int8 weight (see ``int8mm_grouped_weight``)."""

    def __init__(self, buf: torch.Tensor, st: _abi.GroupedWeight):
        self.buf = buf
        self.struct = st
        self.K, self.N, self.G, self.n_keep = st.K, st.N, st.G, st.n_keep

    @property
    def wq(self) -> torch.Tensor:           # N x K int8
        return _view(self.buf, self.struct.wq, self.N * self.K, torch.int8, (self.N, self.K))

    @property
    def col_absmax(self) -> torch.Tensor:   # (K/G) x N float32
        ng = self.K // self.G
        return _view(self.buf, self.struct.col_absmax, ng * self.N, torch.float32, (ng, self.N))

    @property
    def w_keep(self) -> torch.Tensor:
        return _view(self.buf, self.struct.w_keep, self.n_keep * self.N, torch.float16, (self.n_keep, self.N))

    @property
    def keep_idx(self) -> torch.Tensor:
        return _view(self.buf, self.struct.keep_idx, self.n_keep, torch.int32)


def prepare_weight_grouped(W: torch.Tensor, G: int, keep_idx=(), stream=None) -> GroupedWeight:
    """Convert a K x N fp16 CUDA weight to int8 with one constant per output
    column and group of G consecutive k (once, at load)."""
    lib = _abi.load()
    if not (W.is_cuda and W.dtype == torch.float16 and W.dim() == 2 and W.is_contiguous()):
        raise ValueError("W must be a contiguous 2-D float16 CUDA tensor (K x N)")
    K, N = W.shape
    keep = np.unique(np.asarray(keep_idx, dtype=np.int64).ravel()).astype(np.int32)
    nbytes = lib.int8mm_grouped_weight_bytes(K, N, int(G), int(keep.size))
    if nbytes == 0:
        raise Int8mmError(1, f"int8mm_grouped_weight_bytes(K={K}, N={N}, G={G}, n_keep={keep.size})")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    st = _abi.GroupedWeight()
    kp = keep.ctypes.data_as(ctypes.c_void_p) if keep.size else None
    with torch.cuda.device(W.device):
        _abi.check(lib.int8mm_prepare_weight_grouped(ctypes.c_void_p(W.data_ptr()), K, N, int(G), kp, int(keep.size),
                                                     ctypes.c_void_p(buf.data_ptr()), nbytes, ctypes.byref(st),
                                                     _stream(stream)), "int8mm_prepare_weight_grouped")
    return GroupedWeight(buf, st)


def forward_grouped(X: torch.Tensor, w: GroupedWeight, threshold: float = 6.0, *, max_outliers: int | None = None,
                    out: torch.Tensor | None = None, workspace: Workspace | None = None,
                    acc_out: torch.Tensor | None = None, wait_limit_ns: int = 0, test_flags: int = 0,
                    stream=None) -> torch.Tensor:
    """Y = X W by the group-wise method (X: M x K fp16 on the weight's device).
    acc_out (M x N x K/G int32), if given, receives the per-group int32 sums."""
    lib = _abi.load()
    if X.dtype != torch.float16 or X.dim() != 2 or X.shape[1] != w.K or not X.is_cuda or not X.is_contiguous():
        raise ValueError(f"X must be a contiguous float16 CUDA tensor of shape (M, {w.K})")
    M = X.shape[0]
    if workspace is None:
        workspace = Workspace(M, w.K, w.N, max_outliers, device=X.device, G=w.G)
    if (workspace.M, workspace.K, workspace.N, workspace.G) != (M, w.K, w.N, w.G):
        raise ValueError("workspace was made for another shape or group size")
    Y = out if out is not None else torch.empty(M, w.N, dtype=torch.float16, device=X.device)
    opts = _abi.ForwardOpts(0, ctypes.c_void_p(acc_out.data_ptr()) if acc_out is not None else None,
                            int(wait_limit_ns), None, None, int(test_flags))
    with torch.cuda.device(X.device):
        _abi.check(lib.int8mm_forward_grouped(ctypes.c_void_p(X.data_ptr()), M, ctypes.byref(w.struct),
                                              float(threshold), workspace.max_outliers, ctypes.c_void_p(Y.data_ptr()),
                                              ctypes.c_void_p(workspace.buf.data_ptr()), workspace.nbytes,
                                              ctypes.byref(opts), _stream(stream)), "int8mm_forward_grouped")
    return Y


# ---------------------------------------------------------------------------- block-scaled e4m3

_DTYPES = {torch.float16: _abi.F16, torch.bfloat16: _abi.BF16}


_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream  # of a device, as the integer that the C interface takes


def _on(device: torch.device, stream, *used):
    """A context with `device` current, and `stream` if given, so that what a
    call allocates belongs to the stream that it launches on.  `used` (tensors,
    or None) are what the call takes: their memory, which may belong to another
    stream, is not given out again before `stream` is done with it."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    for t in used:
        if t is not None and t.device == device:  # (others are refused by the checks that follow)
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _same_device(what: str, device: torch.device, *tensors) -> None:
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"{what} must be on one device")


def _check_out(t: torch.Tensor, name: str, shape, dtype: torch.dtype, device: torch.device) -> None:
    if (t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def quantize_fp8(X: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                 stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Block-scaled e4m3 codes of a float16 or bfloat16 CUDA matrix: one scale
    per row and 128 consecutive columns (the last block may be shorter).
    Returns (codes float8_e4m3fn M x K, scales float32 M x ceil(K/128)); a
    value is code * scale."""
    if not (X.is_cuda and X.dtype in _DTYPES and X.dim() == 2 and X.is_contiguous()):
        raise ValueError("X must be a contiguous 2-D float16 or bfloat16 CUDA tensor")
    dev = X.device
    if stream is not None or _current_device() != dev.index:
        with _on(dev, stream, X, codes, scales):
            return quantize_fp8(X, codes, scales)
    M, K = X.shape
    kb = (K + 127) // 128
    if codes is None:
        codes = torch.empty_like(X, dtype=torch.float8_e4m3fn)
    else:
        _check_out(codes, "codes", (M, K), torch.float8_e4m3fn, dev)
    if scales is None:
        scales = X.new_empty(M, kb, dtype=torch.float32)
    else:
        _check_out(scales, "scales", (M, kb), torch.float32, dev)
    st = _abi.load().int8mm_quantize_fp8(X.data_ptr(), _DTYPES[X.dtype], M, K, codes.data_ptr(), scales.data_ptr(),
                                         _current_stream(dev.index))
    if st:
        _abi.check(st, "int8mm_quantize_fp8")
    return codes, scales


class Fp8Weight:
    """A block-scaled e4m3 weight (see ``int8mm_fp8_weight`` in the header)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.codes = codes      # N x K float8_e4m3fn
        self.scales = scales    # ceil(N/128) x ceil(K/128) float32
        self.N, self.K = codes.shape
        self.device = codes.device
        self.struct = _abi.Fp8Weight(self.K, self.N, codes.data_ptr(), scales.data_ptr())
        self.ref = ctypes.byref(self.struct)


def _check_codes(what: str, codes: torch.Tensor, scales: torch.Tensor, lead=()) -> None:
    n = len(lead)
    if not (codes.is_cuda and codes.dtype == torch.float8_e4m3fn and codes.dim() == n + 2 and codes.is_contiguous()
            and codes.shape[:n] == torch.Size(lead)):
        raise ValueError(f"{what} codes must be a contiguous float8_e4m3fn CUDA tensor of shape {(*lead, 'N', 'K')}")
    N, K = codes.shape[n:]
    if N < 16 or K < 16 or N % 16 or K % 16:
        raise ValueError(f"{what}: N and K must be multiples of 16, found N={N}, K={K}")
    shape = (*lead, (N + 127) // 128, (K + 127) // 128)
    if scales.dtype != torch.float32 or scales.shape != shape or not scales.is_contiguous():
        raise ValueError(f"{what} scales must be a contiguous float32 tensor of shape {shape}")
    _same_device(f"{what} codes and scales", codes.device, scales)


def weight_fp8(codes: torch.Tensor, scales: torch.Tensor) -> Fp8Weight:
    """The weight whose codes (float8_e4m3fn N x K, one row per output channel)
    and 128 x 128 block scales (float32 ceil(N/128) x ceil(K/128)) the caller
    has, from a block-scaled checkpoint for instance.  Nothing is copied."""
    _check_codes("weight", codes, scales)
    return Fp8Weight(codes, scales)


def prepare_weight_fp8(W: torch.Tensor, stream=None) -> Fp8Weight:
    """Convert a K x N float16 or bfloat16 CUDA weight to e4m3 codes with one
    scale per 128 x 128 block (once, at load)."""
    lib = _abi.load()
    if not (W.is_cuda and W.dtype in _DTYPES and W.dim() == 2 and W.is_contiguous()):
        raise ValueError("W must be a contiguous 2-D float16 or bfloat16 CUDA tensor (K x N)")
    K, N = W.shape
    nbytes = lib.int8mm_fp8_weight_bytes(K, N)
    if nbytes == 0:
        raise Int8mmError(1, f"int8mm_fp8_weight_bytes(K={K}, N={N})")
    st = _abi.Fp8Weight()
    with _on(W.device, stream, W):
        buf = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
        _abi.check(lib.int8mm_prepare_weight_fp8(W.data_ptr(), _DTYPES[W.dtype], K, N, buf.data_ptr(), nbytes,
                                                 ctypes.byref(st), _current_stream(W.device.index)),
                   "int8mm_prepare_weight_fp8")
    nb, kb = (N + 127) // 128, (K + 127) // 128
    return Fp8Weight(_view(buf, st.codes, N * K, torch.float8_e4m3fn, (N, K)),
                     _view(buf, st.scales, nb * kb, torch.float32, (nb, kb)))


class Fp8Workspace:
    """Device scratch of one block-scaled product's shape; zero-filled at
    creation.  Two products that may overlap on the GPU need two of them."""

    def __init__(self, M: int, K: int, N: int, device=None):
        self.M, self.K, self.N = M, K, N
        self.nbytes = _abi.load().int8mm_fp8_workspace_bytes(M, K, N)
        if self.nbytes == 0:
            raise Int8mmError(1, f"int8mm_fp8_workspace_bytes(M={M}, K={K}, N={N})")
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")

    reset = Workspace.reset


def _fp8_opts(path: str, wait_limit_ns: int, test_flags: int):
    if path == "auto" and not wait_limit_ns and not test_flags:
        return None
    return ctypes.byref(_abi.ForwardOpts(_PATHS[path], None, int(wait_limit_ns), None, None, int(test_flags)))


def forward_fp8(X: torch.Tensor, w: Fp8Weight, *, out: torch.Tensor | None = None,
                workspace: Fp8Workspace | None = None, path: str = "auto", wait_limit_ns: int = 0, test_flags: int = 0,
                stream=None) -> torch.Tensor:
    """Y = X W with X (M x K float16 or bfloat16, on the weight's device)
    quantised to e4m3 per row and block of 128 by the call, and the
    block-scaled weight; fp32 sums, Y in X's type.  out must not overlap X.
    path: "auto", "gemm" (tiled) or "decode" (weight-streaming, M <= 1024)."""
    dev = w.device
    if X.dtype not in _DTYPES or X.dim() != 2 or X.shape[1] != w.K or X.device != dev or not X.is_contiguous():
        raise ValueError(f"X must be a contiguous float16 or bfloat16 tensor of shape (M, {w.K}) on {dev}")
    if stream is not None or _current_device() != dev.index:
        with _on(dev, stream, X, w.codes, w.scales, out, workspace and workspace.buf):
            return forward_fp8(X, w, out=out, workspace=workspace, path=path, wait_limit_ns=wait_limit_ns,
                               test_flags=test_flags)
    M = X.shape[0]
    if workspace is None:
        workspace = Fp8Workspace(M, w.K, w.N, device=dev)
    elif (workspace.M, workspace.K, workspace.N) != (M, w.K, w.N) or workspace.buf.device != dev:
        raise ValueError("workspace was made for another shape or device")
    if out is None:
        out = X.new_empty(M, w.N)
    else:
        _check_out(out, "out", (M, w.N), X.dtype, dev)
    st = _abi.load().int8mm_forward_fp8(X.data_ptr(), _DTYPES[X.dtype], M, w.ref, out.data_ptr(),
                                        workspace.buf.data_ptr(), workspace.nbytes,
                                        _fp8_opts(path, wait_limit_ns, test_flags), _current_stream(dev.index))
    if st:
        _abi.check(st, "int8mm_forward_fp8")
    return out


# ---------------------------------------------------------------------------- mixture of experts

class MoeFp8Weight:
    """The weights of a mixture-of-experts feed-forward layer (see
    ``int8mm_moe_weight`` in the header)."""

    def __init__(self, router: torch.Tensor, gate, up, down):
        self.router, self.gate, self.up, self.down = router, gate, up, down
        self.E, self.I, self.H = gate[0].shape
        self.device = router.device
        self.struct = _abi.MoeWeight(self.E, self.H, self.I, router.data_ptr(),
                                     *(t.data_ptr() for pair in (gate, up, down) for t in pair))
        self.ref = ctypes.byref(self.struct)


def moe_weight_fp8(router: torch.Tensor, gate, up, down) -> MoeFp8Weight:
    """The layer of E experts y = (silu(x Wg) * (x Wu)) Wd from weights that
    are block-scaled e4m3 already.  router: E x H float16 or bfloat16 (the type
    of the layer's X); gate, up: (codes float8_e4m3fn E x I x H, scales float32
    E x ceil(I/128) x ceil(H/128)); down: (codes E x H x I, scales).  Nothing
    is copied."""
    if not (router.is_cuda and router.dtype in _DTYPES and router.dim() == 2 and router.is_contiguous()):
        raise ValueError("router must be a contiguous 2-D float16 or bfloat16 CUDA tensor (E x H)")
    E, H = router.shape
    gate, up, down = tuple(gate), tuple(up), tuple(down)
    for what, (codes, scales) in (("gate", gate), ("up", up), ("down", down)):
        _check_codes(what, codes, scales, (E,))
    inner = gate[0].shape[1]
    if gate[0].shape != (E, inner, H) or up[0].shape != (E, inner, H) or down[0].shape != (E, H, inner):
        raise ValueError("gate and up must be E x I x H and down E x H x I, with the router's E and H")
    _same_device("the layer's weights", router.device, gate[0], up[0], down[0])
    return MoeFp8Weight(router, gate, up, down)


def prepare_moe_weight_fp8(router: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor,
                           stream=None) -> MoeFp8Weight:
    """Convert a layer's 16-bit weights once (at load): router E x H; gate and
    up E x H x I, down E x I x H (each expert K x N, as prepare_weight_fp8
    takes it), float16 or bfloat16 CUDA tensors."""
    for what, W in (("gate", gate), ("up", up), ("down", down)):
        if not (W.is_cuda and W.dtype in _DTYPES and W.dim() == 3 and W.is_contiguous()):
            raise ValueError(f"{what} must be a contiguous 3-D float16 or bfloat16 CUDA tensor")

    def convert(W):
        parts = [prepare_weight_fp8(We, stream) for We in W]
        with _on(W.device, stream):
            return torch.stack([q.codes for q in parts]), torch.stack([q.scales for q in parts])

    return moe_weight_fp8(router, convert(gate), convert(up), convert(down))


class MoeWorkspace:
    """Device scratch of a mixture-of-experts layer for T tokens; zero-filled
    at creation.  Two calls that may overlap on the GPU need two of them."""

    def __init__(self, T: int, w: MoeFp8Weight, top_k: int, device=None):
        self.T, self.H, self.I, self.E, self.top_k = T, w.H, w.I, w.E, top_k
        self.nbytes = _abi.load().int8mm_moe_workspace_bytes(T, w.H, w.I, w.E, top_k)
        if self.nbytes == 0:
            raise Int8mmError(1, f"int8mm_moe_workspace_bytes(T={T}, H={w.H}, I={w.I}, E={w.E}, top_k={top_k})")
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or w.router.device)

    reset = Workspace.reset


def forward_moe_fp8(X: torch.Tensor, w: MoeFp8Weight, top_k: int, *, renormalize: bool = True,
                    out: torch.Tensor | None = None, workspace: MoeWorkspace | None = None,
                    return_routing: bool = False, wait_limit_ns: int = 0, test_flags: int = 0, stream=None):
    """The mixture-of-experts layer on a few tokens: X is T x H (T <= 64) in the
    router's type and on its device.  Each token takes the top_k experts of
    softmax(X router^T), ties to the lower index, with those probabilities as
    weights (renormalize: divided by their sum); out may be X.  Returns Y, T x H
    in X's type, and with return_routing also the experts (int32 T x top_k, best
    first) and their weights (float32 T x top_k)."""
    dev = w.device
    if X.dtype != w.router.dtype or X.dim() != 2 or X.shape[1] != w.H or X.device != dev or not X.is_contiguous():
        raise ValueError(f"X must be a contiguous {w.router.dtype} tensor of shape (T, {w.H}) on {dev}")
    if stream is not None or _current_device() != dev.index:
        with _on(dev, stream, X, w.router, *w.gate, *w.up, *w.down, out, workspace and workspace.buf):
            return forward_moe_fp8(X, w, top_k, renormalize=renormalize, out=out, workspace=workspace,
                                   return_routing=return_routing, wait_limit_ns=wait_limit_ns, test_flags=test_flags)
    T = X.shape[0]
    if workspace is None:
        workspace = MoeWorkspace(T, w, top_k)
    elif ((workspace.T, workspace.H, workspace.I, workspace.E, workspace.top_k) != (T, w.H, w.I, w.E, top_k)
          or workspace.buf.device != dev):
        raise ValueError("workspace was made for another shape or device")
    if out is None:
        out = X.new_empty(T, w.H)
    else:
        _check_out(out, "out", (T, w.H), X.dtype, dev)
    ids = wts = None
    if return_routing:
        ids = X.new_empty(T, top_k, dtype=torch.int32)
        wts = X.new_empty(T, top_k, dtype=torch.float32)
    st = _abi.load().int8mm_forward_moe_fp8(
        X.data_ptr(), _DTYPES[X.dtype], T, w.ref, top_k, int(bool(renormalize)), out.data_ptr(),
        ids.data_ptr() if return_routing else None, wts.data_ptr() if return_routing else None,
        workspace.buf.data_ptr(), workspace.nbytes, _fp8_opts("auto", wait_limit_ns, test_flags),
        _current_stream(dev.index))
    if st:
        _abi.check(st, "int8mm_forward_moe_fp8")
    return (out, ids, wts) if return_routing else out
