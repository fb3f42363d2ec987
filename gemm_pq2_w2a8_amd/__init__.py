"""Thin Python binding of the PQ2_0 C ABI (include/pq2.h), for PyTorch tensors.

Argument marshalling only: tensors are checked for dtype, shape, device and
contiguity, their device pointers and the current HIP stream are passed to
``libpq2.so``, and a non-zero status raises :class:`PQ2Error`. Every step of
the computation runs in the library's gfx950 kernels; there is no fallback.
Importing this package raises if ``libpq2.so`` has not been built
(``python gemm_pq2_w2a8_amd/build.py``).
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpq2.so")

GROUP = 128
PATH_AUTO, PATH_GEMV, PATH_SMALL, PATH_PREFILL, PATH_PANEL = 0, 1, 2, 3, 4
ACT_F32, ACT_BF16, ACT_F16 = 0, 1, 2

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python gemm_pq2_w2a8_amd/build.py`")

lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
lib.pq2_abi_version.restype = ctypes.c_int
lib.pq2_abi_version.argtypes = []
lib.pq2_status_str.restype = ctypes.c_char_p
lib.pq2_status_str.argtypes = [ctypes.c_int]
lib.pq2_quantize_act.restype = ctypes.c_int
lib.pq2_quantize_act.argtypes = [_P, _P, _P, _P, _I64, _I64, _P]
lib.pq2_quantize_act_16.restype = ctypes.c_int
lib.pq2_quantize_act_16.argtypes = [_P, ctypes.c_int, _P, _P, _P, _I64, _I64, _P]
_F32 = ctypes.c_float
lib.pq2_norm_quantize.restype = ctypes.c_int
lib.pq2_norm_quantize.argtypes = [_P, ctypes.c_int, _P, _P, _P, _I64, _F32, _P, _F32, _P, _P, _P,
                                  _P, _P, _I64, _I64, _P]
_SZ = ctypes.c_size_t
lib.pq2_gemm_workspace_bytes.restype = _SZ
lib.pq2_gemm_workspace_bytes.argtypes = [_I64, _I64, _I64]
lib.pq2_gemm.restype = ctypes.c_int
lib.pq2_gemm.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]
lib.pq2_gemm_bf16.restype = ctypes.c_int
lib.pq2_gemm_bf16.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]
lib.pq2_gemm_noalloc.restype = ctypes.c_int
lib.pq2_gemm_noalloc.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]
lib.pq2_gemm_kernel_path.restype = ctypes.c_int
lib.pq2_gemm_kernel_path.argtypes = [_I64, _I64, _I64, _SZ]
lib.pq2_gemm_path.restype = ctypes.c_int
lib.pq2_gemm_path.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P, _SZ,
                              _P]
lib.pq2_gemm_group_dots.restype = ctypes.c_int
lib.pq2_gemm_group_dots.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P]
lib.pq2_gemm_grouped.restype = ctypes.c_int
lib.pq2_gemm_grouped.argtypes = [_P, _P, _P, _I64, _P, _P, _P, _I64, _P, _P, _P, ctypes.c_int,
                                 _I64, _I64, _I64, _P]
lib.pq2_lora_add.restype = ctypes.c_int
lib.pq2_lora_add.argtypes = [_P, ctypes.c_int, _P, _P, ctypes.c_int, _P, _P, _P, _P, _P,
                             ctypes.c_int, _I64, _I64, _I64, _I64, _I64, _P, _SZ, _P]
lib.pq2_lora_workspace_bytes.restype = _SZ
lib.pq2_lora_workspace_bytes.argtypes = [_I64, _I64, _I64]
lib.pq2_linear.restype = ctypes.c_int
lib.pq2_linear.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]
lib.pq2_linear_workspace_bytes.restype = _SZ
lib.pq2_linear_workspace_bytes.argtypes = [_I64, _I64, _I64]
lib.pq2_linear_kernel_path.restype = ctypes.c_int
lib.pq2_linear_kernel_path.argtypes = [_I64, _I64, _I64, _SZ]

LINEAR_MAX_M = 16   # PQ2_LINEAR_MAX_M

# Every extern "C" symbol declared in include/pq2.h.
ABI_SYMBOLS = ("pq2_abi_version", "pq2_status_str", "pq2_quantize_act", "pq2_quantize_act_16",
               "pq2_norm_quantize", "pq2_gemm_grouped", "pq2_lora_add", "pq2_lora_workspace_bytes",
               "pq2_gemm_workspace_bytes", "pq2_gemm", "pq2_gemm_noalloc", "pq2_gemm_bf16",
               "pq2_gemm_kernel_path", "pq2_gemm_path", "pq2_linear", "pq2_linear_workspace_bytes",
               "pq2_linear_kernel_path", "pq2_gemm_group_dots")

NOALLOC_SCRATCH_BYTES = 16 << 20    # PQ2_NOALLOC_SCRATCH_BYTES

PATH_NAMES = {PATH_GEMV: "gemv_dot4", PATH_SMALL: "small_mfma", PATH_PREFILL: "prefill_mfma",
              PATH_PANEL: "small_panel"}


def gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes of pq2_gemm's fastest plan for this shape (0: none needed)."""
    return int(lib.pq2_gemm_workspace_bytes(M, N, K))


def linear_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes of pq2_linear's plan for this shape (0: none needed)."""
    return int(lib.pq2_linear_workspace_bytes(M, N, K))


def lora_workspace_bytes(M: int, K: int, R: int) -> int:
    """Workspace bytes of pq2_lora_add's fastest plan for this shape."""
    return int(lib.pq2_lora_workspace_bytes(M, K, R))


def linear_kernel_path(M: int, N: int, K: int, workspace_bytes: Optional[int] = None) -> int:
    """PATH_GEMV or PATH_PANEL: the kernel pq2_linear takes for this shape given
    a workspace of that many bytes (None: what linear_workspace_bytes asks
    for); -1 where pq2_linear rejects the shape."""
    if workspace_bytes is None:
        workspace_bytes = linear_workspace_bytes(M, N, K)
    return int(lib.pq2_linear_kernel_path(M, N, K, int(workspace_bytes)))


def gemm_kernel_path(M: int, N: int, K: int, workspace_bytes: Optional[int] = None) -> int:
    """PATH_* that pq2_gemm takes for this shape on the current device given a
    workspace of that many bytes (None: the size gemm_workspace_bytes asks
    for); -1 for a bad shape."""
    if workspace_bytes is None:
        workspace_bytes = gemm_workspace_bytes(M, N, K)
    return int(lib.pq2_gemm_kernel_path(M, N, K, int(workspace_bytes)))


class PQ2Error(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(lib.pq2_status_str(status).decode())


def _check(status: int) -> None:
    if status != 0:
        raise PQ2Error(status)


def abi_version() -> int:
    return int(lib.pq2_abi_version())


def _handle(stream, index: int) -> int:
    """Handle of a stream argument; ValueError for a stream of another GPU than
    the tensors' (a raw handle does not tell)."""
    if not isinstance(stream, torch.cuda.Stream):
        return int(stream)
    if stream.device_index != index:
        raise ValueError(f"stream must be on cuda:{index}, got cuda:{stream.device_index}")
    return stream.cuda_stream


def _stream(t: torch.Tensor, stream) -> int:
    if stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return _handle(stream, t.get_device())


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: Tuple[int, ...]) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: Tuple[int, ...],
         index: int) -> int:
    """Address of a contiguous tensor of this type and shape on GPU `index` (0 for
    None); raises what _need raises, and ValueError for another GPU."""
    if t is None:
        return 0
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == index and t.is_contiguous()):
        _need(t, name, dtype, shape)
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    return t.data_ptr()


def _gpu(t: torch.Tensor, name: str) -> int:
    """Index of the GPU a tensor is on."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return index


def _launch(index: int, stream, call, *args) -> None:
    """call(*args, stream) on GPU `index`: a kernel runs on the current device,
    which need not be the tensors'."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        raw = _handle(stream, index)
    if torch._C._cuda_getDevice() == index:
        _check(call(*args, raw))
        return
    with torch.cuda.device(index):
        _check(call(*args, raw))


_ACT_FORMAT = {torch.float32: ACT_F32, torch.bfloat16: ACT_BF16, torch.float16: ACT_F16}


def _format(x: torch.Tensor, name: str) -> int:
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    fmt = _ACT_FORMAT.get(x.dtype)
    if fmt is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {x.dtype}")
    return fmt


def _mk(x: torch.Tensor) -> Tuple[int, int]:
    if x.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    return int(x.shape[0]), int(x.shape[1])


def pq2_quantize_act(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, t: torch.Tensor,
                     stream=None) -> None:
    """x float32, bfloat16 or float16 [M][K] -> q int8 [M][K] (plane order),
    s float32 [M][G], t int32 [M][G]; 16-bit x is widened exactly first."""
    M, K = _mk(x)
    G = K // GROUP
    _need(q, "q", torch.int8, (M, K))
    _need(s, "s", torch.float32, (M, G))
    _need(t, "t", torch.int32, (M, G))
    if x.dtype in (torch.bfloat16, torch.float16):
        _need(x, "x", x.dtype, (M, K))
        fmt = ACT_BF16 if x.dtype == torch.bfloat16 else ACT_F16
        _check(lib.pq2_quantize_act_16(x.data_ptr(), fmt, q.data_ptr(), s.data_ptr(),
                                       t.data_ptr(), M, K, _stream(x, stream)))
        return
    _need(x, "x", torch.float32, (M, K))
    _check(lib.pq2_quantize_act(x.data_ptr(), q.data_ptr(), s.data_ptr(), t.data_ptr(), M, K,
                                _stream(x, stream)))


def pq2_norm_quantize(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                      s: Optional[torch.Tensor] = None, t: Optional[torch.Tensor] = None, *,
                      residual: Optional[torch.Tensor] = None,
                      w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                      alpha: float = 1.0, w_pre: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      h: Optional[torch.Tensor] = None, n: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """The norms after and before a block with its gate and residual scale,
    ending in the quantiser:

        h = residual + alpha * gate * (rms(x) * w_post),   n = rms(h) * w_pre,
        q, s, t = pq2_quantize_act's of n

    x, residual, h, n [M][K] and gate [rows][K] (rows dividing M; [K] is one
    row) share x's type (float32, bfloat16 or float16); w_post, w_pre float32
    [K]; q, s, t as for pq2_quantize_act, all or none. Whatever is None is left
    out; h may be residual or x."""
    fmt = _format(x, "x")
    M, K = _mk(x)
    G = K // GROUP
    ty, at = x.dtype, _gpu(x, "x")
    gate_rows = 0
    if gate is not None:
        if not isinstance(gate, torch.Tensor) or gate.dim() not in (1, 2):
            raise ValueError("gate must be a 1-D or 2-D tensor")
        gate_rows = 1 if gate.dim() == 1 else int(gate.shape[0])
        gate = gate.view(1, -1) if gate.dim() == 1 else gate
    mk = (M, K)
    _launch(at, stream, lib.pq2_norm_quantize, _ptr(x, "x", ty, mk, at), fmt,
            _ptr(residual, "residual", ty, mk, at), _ptr(w_post, "w_post", torch.float32, (K,), at),
            _ptr(gate, "gate", ty, (gate_rows, K), at), gate_rows, alpha,
            _ptr(w_pre, "w_pre", torch.float32, (K,), at), eps, _ptr(h, "h", ty, mk, at),
            _ptr(n, "n", ty, mk, at), _ptr(q, "q", torch.int8, mk, at),
            _ptr(s, "s", torch.float32, (M, G), at), _ptr(t, "t", torch.int32, (M, G), at), M, K)


_CURRENT = contextlib.nullcontext()


def _on(stream, device):
    """Context in which torch allocates from the pool of the stream that a call is
    launched on: a block of another stream's pool may have work pending there
    that nothing orders before the call."""
    if stream is None:
        return _CURRENT
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else
                             torch.cuda.ExternalStream(int(stream), device=device))


def _workspace(workspace, M: int, N: int, K: int, device, stream,
               query=None) -> Tuple[int, int, object]:
    """(pointer, bytes, keep-alive) of the split-K workspace argument: "auto"
    allocates the size pq2_gemm_workspace_bytes (or `query`) asks for with
    torch (none when 0), None passes no workspace, a device tensor passes its storage. An
    "auto" buffer comes from the launch stream's pool: its earlier uses and its
    next ones are on that stream too, and so in order with this call's."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be "auto", None or a device tensor')
        n = (query or gemm_workspace_bytes)(M, N, K)
        if n == 0:
            return 0, 0, None
        if stream is None:
            workspace = torch.empty(n, dtype=torch.uint8, device=device)
        else:
            with _on(stream, device):
                workspace = torch.empty(n, dtype=torch.uint8, device=device)
    if workspace is None:
        return 0, 0, None
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise ValueError("workspace must be a GPU tensor")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def pq2_gemm(q: torch.Tensor, s: torch.Tensor, t: torch.Tensor, codes: torch.Tensor,
             wscale: torch.Tensor, y: torch.Tensor, workspace="auto", stream=None) -> None:
    """y [M][N] = PQ2_0 product of plane-order q/s/t and codes/wscale; y float32,
    or bfloat16 (pq2_gemm_bf16: the float32 result rounded to nearest-even).
    workspace: "auto" (torch allocates what the fastest plan needs), None (no
    workspace: plans that do not split K) or a device tensor."""
    M, K = _mk(q)
    N = int(codes.shape[0])
    G = K // GROUP
    _need(q, "q", torch.int8, (M, K))
    _need(s, "s", torch.float32, (M, G))
    _need(t, "t", torch.int32, (M, G))
    _need(codes, "codes", torch.uint8, (N, K // 4))
    if wscale.dtype == torch.float16:
        wscale = wscale.view(torch.int16)
    _need(wscale, "wscale", torch.int16, (N, G))
    wp, wn, _keep = _workspace(workspace, M, N, K, q.device, stream)
    if y.dtype == torch.bfloat16:
        _need(y, "y", torch.bfloat16, (M, N))
        _check(lib.pq2_gemm_bf16(q.data_ptr(), s.data_ptr(), t.data_ptr(), codes.data_ptr(),
                                 wscale.data_ptr(), y.data_ptr(), M, N, K, wp, wn,
                                 _stream(q, stream)))
        return
    _need(y, "y", torch.float32, (M, N))
    _check(lib.pq2_gemm(q.data_ptr(), s.data_ptr(), t.data_ptr(), codes.data_ptr(),
                        wscale.data_ptr(), y.data_ptr(), M, N, K, wp, wn, _stream(q, stream)))


def pq2_gemm_noalloc(q: torch.Tensor, s: torch.Tensor, t: torch.Tensor, codes: torch.Tensor,
                     wscale: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """pq2_gemm with the library's own per-device split-K scratch: no workspace,
    no allocation (calls that overlap on one device race on the scratch)."""
    M, K = _mk(q)
    N = int(codes.shape[0])
    G = K // GROUP
    _need(q, "q", torch.int8, (M, K))
    _need(s, "s", torch.float32, (M, G))
    _need(t, "t", torch.int32, (M, G))
    _need(codes, "codes", torch.uint8, (N, K // 4))
    if wscale.dtype == torch.float16:
        wscale = wscale.view(torch.int16)
    _need(wscale, "wscale", torch.int16, (N, G))
    _need(y, "y", torch.float32, (M, N))
    _check(lib.pq2_gemm_noalloc(q.data_ptr(), s.data_ptr(), t.data_ptr(), codes.data_ptr(),
                                wscale.data_ptr(), y.data_ptr(), M, N, K, _stream(q, stream)))


def pq2_gemm_path(q: torch.Tensor, s: torch.Tensor, t: torch.Tensor, codes: torch.Tensor,
                  wscale: torch.Tensor, y: torch.Tensor, path: int, workspace="auto",
                  stream=None) -> None:
    """pq2_gemm through the selected kernel path (PATH_*); workspace as for pq2_gemm."""
    M, K = _mk(q)
    N = int(codes.shape[0])
    G = K // GROUP
    _need(q, "q", torch.int8, (M, K))
    _need(s, "s", torch.float32, (M, G))
    _need(t, "t", torch.int32, (M, G))
    _need(codes, "codes", torch.uint8, (N, K // 4))
    if wscale.dtype == torch.float16:
        wscale = wscale.view(torch.int16)
    _need(wscale, "wscale", torch.int16, (N, G))
    _need(y, "y", torch.float32, (M, N))
    wp, wn, _keep = _workspace(workspace, M, N, K, q.device, stream)
    _check(lib.pq2_gemm_path(q.data_ptr(), s.data_ptr(), t.data_ptr(), codes.data_ptr(),
                             wscale.data_ptr(), y.data_ptr(), M, N, K, int(path), wp, wn,
                             _stream(q, stream)))


def pq2_gemm_grouped(q: torch.Tensor, s: torch.Tensor, t: torch.Tensor, codes: torch.Tensor,
                     wscale: torch.Tensor, offsets: torch.Tensor, y: torch.Tensor,
                     rows: Optional[torch.Tensor] = None,
                     row_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """y [T][N] (float32 or bfloat16): slot i of expert e (offsets[e] <= i <
    offsets[e + 1]) = row_scale[i] * the PQ2_0 product of activation row rows[i]
    of plane-order q/s/t [R] and codes[e], wscale[e].

    codes uint8 [E][N][K/4], wscale [E][N][G], offsets int32 [E + 1] on the
    device, rows int32 [T] (None: row i; a row outside [0, R) gives zeros),
    row_scale float32 [T] or None. Slots behind offsets[E] are left alone."""
    R, K = _mk(q)
    G = K // GROUP
    if codes.dim() != 3 or y.dim() != 2:
        raise ValueError("expected 3-D codes and 2-D y")
    E, N, T = int(codes.shape[0]), int(codes.shape[1]), int(y.shape[0])
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"y must be float32 or bfloat16, got {y.dtype}")
    at = _gpu(q, "q")
    if wscale.dtype == torch.float16:
        wscale = wscale.view(torch.int16)
    _launch(at, stream, lib.pq2_gemm_grouped, _ptr(q, "q", torch.int8, (R, K), at),
            _ptr(s, "s", torch.float32, (R, G), at), _ptr(t, "t", torch.int32, (R, G), at), R,
            _ptr(codes, "codes", torch.uint8, (E, N, K // 4), at),
            _ptr(wscale, "wscale", torch.int16, (E, N, G), at),
            _ptr(offsets, "offsets", torch.int32, (E + 1,), at), E,
            _ptr(rows, "rows", torch.int32, (T,), at),
            _ptr(row_scale, "row_scale", torch.float32, (T,), at), _ptr(y, "y", y.dtype, (T, N), at),
            _ACT_FORMAT[y.dtype], T, N, K)


def pq2_lora_add(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, adapter: torch.Tensor,
                 y: torch.Tensor, base: Optional[torch.Tensor] = None,
                 ranks: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                 workspace="auto", stream=None) -> None:
    """y[m] = base[m] + scale[l] * b[l] @ (a[l] @ x[m]) with l = adapter[m]; rows
    whose adapter is outside [0, L) copy their base.

    x [M][K] float32, bfloat16 or float16; a [L][R][K], b [L][N][R] bfloat16 or
    float16; adapter int32 [M]; ranks int32 [L] (None: R), scale float32 [L]
    (None: 1); y and base [M][N] float32 or bfloat16, base None or y itself for
    an addition in place. workspace: "auto" (torch allocates) or a device
    tensor of lora_workspace_bytes(M, K, R) bytes (at least M * R floats)."""
    fmt = _format(x, "x")
    M, K = _mk(x)
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("expected 3-D a and b")
    if a.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"a must be bfloat16 or float16, got {a.dtype}")
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"y must be float32 or bfloat16, got {y.dtype}")
    at = _gpu(x, "x")
    L, R, N = int(a.shape[0]), int(a.shape[1]), int(b.shape[1])
    args = (_ptr(x, "x", x.dtype, (M, K), at), fmt, _ptr(a, "a", a.dtype, (L, R, K), at),
            _ptr(b, "b", a.dtype, (L, N, R), at), _ACT_FORMAT[a.dtype],
            _ptr(adapter, "adapter", torch.int32, (M,), at), _ptr(ranks, "ranks", torch.int32, (L,), at),
            _ptr(scale, "scale", torch.float32, (L,), at), _ptr(base, "base", y.dtype, (M, N), at),
            _ptr(y, "y", y.dtype, (M, N), at), _ACT_FORMAT[y.dtype], M, N, K, R, L)
    wp, wn, keep = _workspace(workspace, M, K, R, x.device, stream, lora_workspace_bytes)
    if keep is not None and keep.get_device() != at:
        raise ValueError(f"workspace must be on cuda:{at}, got {keep.device}")
    _launch(at, stream, lib.pq2_lora_add, *args, wp, wn)


def pq2_linear(x: torch.Tensor, codes: torch.Tensor, wscale: torch.Tensor, y: torch.Tensor,
               workspace="auto", stream=None) -> None:
    """y float32 [M][N] from float32 x [M][K] with the quantisation inside the
    GEMM kernel (M <= LINEAR_MAX_M). workspace as for pq2_gemm, sized by
    linear_workspace_bytes."""
    M, K = _mk(x)
    N = int(codes.shape[0])
    G = K // GROUP
    _need(x, "x", torch.float32, (M, K))
    _need(codes, "codes", torch.uint8, (N, K // 4))
    if wscale.dtype == torch.float16:
        wscale = wscale.view(torch.int16)
    _need(wscale, "wscale", torch.int16, (N, G))
    _need(y, "y", torch.float32, (M, N))
    wp, wn, _keep = _workspace(workspace, M, N, K, x.device, stream, linear_workspace_bytes)
    _check(lib.pq2_linear(x.data_ptr(), codes.data_ptr(), wscale.data_ptr(), y.data_ptr(),
                          M, N, K, wp, wn, _stream(x, stream)))


def pq2_gemm_group_dots(q: torch.Tensor, t: torch.Tensor, codes: torch.Tensor,
                        d: torch.Tensor, path: int = PATH_AUTO, stream=None) -> None:
    """d int32 [M][N][G] = exact group dots through the selected kernel path."""
    M, K = _mk(q)
    N = int(codes.shape[0])
    G = K // GROUP
    _need(q, "q", torch.int8, (M, K))
    _need(t, "t", torch.int32, (M, G))
    _need(codes, "codes", torch.uint8, (N, K // 4))
    _need(d, "d", torch.int32, (M, N, G))
    _check(lib.pq2_gemm_group_dots(q.data_ptr(), t.data_ptr(), codes.data_ptr(), d.data_ptr(),
                                   M, N, K, int(path), _stream(q, stream)))


# ---------------------------------------------------------------- allocating helpers

def _returned(stream, *tensors: torch.Tensor):
    """The tensors, recorded on the caller's stream where they come from the pool
    of another: their memory is not used again before what the caller enqueues
    there while holding them is done."""
    if stream is not None:
        for t in tensors:
            t.record_stream(torch.cuda.current_stream(t.device))
    return tensors


def _qst(M: int, K: int, device) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    return (torch.empty((M, K), dtype=torch.int8, device=device),
            torch.empty((M, K // GROUP), dtype=torch.float32, device=device),
            torch.empty((M, K // GROUP), dtype=torch.int32, device=device))


def quantize_act(x: torch.Tensor, stream=None):
    """Allocate q/s/t with torch (from the launch stream's pool) and run
    pq2_quantize_act."""
    M, K = _mk(x)
    with _on(stream, x.device):
        q, s, t = _qst(M, K, x.device)
    pq2_quantize_act(x, q, s, t, stream)
    return _returned(stream, q, s, t)


def norm_quantize(x: torch.Tensor, *, residual: Optional[torch.Tensor] = None,
                  w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  alpha: float = 1.0, w_pre: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  stream=None):
    """Allocate h and q/s/t with torch (from the launch stream's pool) and run
    pq2_norm_quantize: (h, q, s, t)."""
    _format(x, "x")
    M, K = _mk(x)
    with _on(stream, x.device):
        h = torch.empty_like(x)
        q, s, t = _qst(M, K, x.device)
    pq2_norm_quantize(x, q, s, t, residual=residual, w_post=w_post, gate=gate, alpha=alpha,
                      w_pre=w_pre, eps=eps, h=h, stream=stream)
    return _returned(stream, h, q, s, t)


def linear(x: torch.Tensor, codes: torch.Tensor, wscale: torch.Tensor,
           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Whole path, y float32 [M][N]: pq2_linear for float32 x with one token
    row (where quantising inside the GEMV beats the separate launch), else
    pq2_quantize_act (float32, bfloat16 or float16 x) into torch-allocated
    q/s/t followed by pq2_gemm."""
    M, K = _mk(x)
    N = int(codes.shape[0])
    fused = M == 1 and x.dtype == torch.float32
    with _on(stream, x.device):
        y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=x.device)
        q, s, t = (None, None, None) if fused else _qst(M, K, x.device)
    if fused:
        pq2_linear(x, codes, wscale, y, stream=stream)
    else:
        pq2_quantize_act(x, q, s, t, stream)
        pq2_gemm(q, s, t, codes, wscale, y, stream=stream)
    if out is None:
        _returned(stream, y)
    return y
