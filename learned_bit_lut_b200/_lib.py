"""ctypes binding of libany4.so (include/any4.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, and their device pointers plus the current CUDA stream are passed
to the C ABI. Every step of the computation runs in the library's kernels;
there is no fallback path. Importing this module fails loudly when the
library has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libany4.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python learned_bit_lut_b200/build.py`")

lib = ctypes.CDLL(LIB_PATH)

_c_size = ctypes.c_size_t
_c_int = ctypes.c_int
_p = ctypes.c_void_p

lib.any4_packed_bytes.argtypes = [_c_int, _c_int, _c_int]
lib.any4_packed_bytes.restype = _c_size
lib.any4_pack.argtypes = [_p, _p, _p, _p, _c_int, _c_int, _c_int, _p, _c_size, _p]
lib.any4_pack.restype = _c_int
lib.any4_dequant.argtypes = [_p, _c_int, _c_int, _c_int, _p, _p]
lib.any4_dequant.restype = _c_int
lib.any4_linear_workspace_bytes.argtypes = [_c_int, _c_int, _c_int, _c_int]
lib.any4_linear_workspace_bytes.restype = _c_size
lib.any4_linear_workspace_bytes_bits.argtypes = [_c_int, _c_int, _c_int, _c_int, _c_int]
lib.any4_linear_workspace_bytes_bits.restype = _c_size
lib.any4_linear_grid.argtypes = [_c_int, _c_int, _c_int, _c_int, _c_int, _p, _p]
lib.any4_linear_grid.restype = _c_int
lib.any4_linear_kernel.argtypes = [_c_int, _c_int, _c_int, _c_int, _c_int]
lib.any4_linear_kernel.restype = _c_int
lib.any4_linear.argtypes = [_p, _p, _c_int, _c_int, _c_int, _c_int, _p, _p, _c_size, _p]
lib.any4_linear.restype = _c_int
lib.any4_linear_noalloc.argtypes = [_p, _p, _c_int, _c_int, _c_int, _c_int, _p, _p]
lib.any4_linear_noalloc.restype = _c_int
lib.any4_noalloc_status_word.argtypes = [ctypes.POINTER(_p)]
lib.any4_noalloc_status_word.restype = _c_int
lib.any4_format_lut.argtypes = [_c_int, _p]
lib.any4_format_lut.restype = _c_int
lib.any4_pack_format.argtypes = [_c_int, _p, _p, _p, _c_int, _c_int, _c_int, _p, _c_size, _p]
lib.any4_pack_format.restype = _c_int
lib.any4_quantize.argtypes = [_p, _p, _c_int, _c_int, _c_int, _c_int, _c_int, _p, _p, _p, _p, _p]
lib.any4_quantize.restype = _c_int
lib.any4_packed_bytes_bits.argtypes = [_c_int, _c_int, _c_int, _c_int]
lib.any4_packed_bytes_bits.restype = _c_size
lib.any4_pack_bits.argtypes = [_c_int, _p, _p, _p, _p, _c_int, _c_int, _c_int, _p, _c_size, _p]
lib.any4_pack_bits.restype = _c_int
lib.any4_dequant_bits.argtypes = [_c_int, _p, _c_int, _c_int, _c_int, _p, _p]
lib.any4_dequant_bits.restype = _c_int
lib.any4_linear_bits.argtypes = [_c_int, _p, _p, _c_int, _c_int, _c_int, _c_int, _p, _p, _c_size, _p]
lib.any4_linear_bits.restype = _c_int
lib.any4_lora_header_bytes.argtypes = []
lib.any4_lora_header_bytes.restype = _c_size
lib.any4_lora_workspace_bytes.argtypes = [_c_int] * 7
lib.any4_lora_workspace_bytes.restype = _c_size
lib.any4_linear_lora.argtypes = [_c_int, _p, _p, _c_int, _c_int, _c_int, _c_int, _p, _p, _p, _p, _c_int, _c_int,
                                 _p, _p, _p, _c_size, _p]
lib.any4_linear_lora.restype = _c_int
lib.any4_lora_grad_workspace_bytes.argtypes = [_c_int] * 7
lib.any4_lora_grad_workspace_bytes.restype = _c_size
lib.any4_linear_lora_grad.argtypes = [_c_int, _p, _p, _p, _p, _c_int, _p, _p, _c_int, _c_int, _c_int, _c_int,
                                      _p, _p, _p, _p, _c_int, _c_int, _p, _p, _p, _p, _c_size, _p]
lib.any4_linear_lora_grad.restype = _c_int
lib.any4_act_pack.argtypes = [_p, _c_int, _c_int, _c_int, _p, _p, _p]
lib.any4_act_pack.restype = _c_int
lib.any4_act_unpack.argtypes = [_p, _p, _c_int, _c_int, _c_int, _p, _p]
lib.any4_act_unpack.restype = _c_int
lib.any4_stream_capture_id.argtypes = [_p, ctypes.POINTER(ctypes.c_uint64)]
lib.any4_stream_capture_id.restype = _c_int
lib.any4_strerror.argtypes = [_c_int]
lib.any4_strerror.restype = ctypes.c_char_p
lib.any4_last_cuda_error.argtypes = []
lib.any4_last_cuda_error.restype = _c_int

EXPORTED = ("any4_packed_bytes", "any4_pack", "any4_dequant", "any4_linear_workspace_bytes",
            "any4_linear_workspace_bytes_bits", "any4_linear_grid", "any4_linear_kernel",
            "any4_linear", "any4_linear_noalloc", "any4_noalloc_status_word", "any4_quantize", "any4_format_lut",
            "any4_pack_format", "any4_packed_bytes_bits", "any4_pack_bits", "any4_dequant_bits",
            "any4_linear_bits", "any4_lora_header_bytes", "any4_lora_workspace_bytes", "any4_linear_lora",
            "any4_lora_grad_workspace_bytes", "any4_linear_lora_grad", "any4_act_pack", "any4_act_unpack",
            "any4_stream_capture_id", "any4_strerror", "any4_last_cuda_error")

ANY4_FORMAT_INT4, ANY4_FORMAT_NF4, ANY4_FORMAT_FP4 = 1, 2, 3
FORMATS = {"int4": ANY4_FORMAT_INT4, "nf4": ANY4_FORMAT_NF4, "fp4": ANY4_FORMAT_FP4}

ANY4_OK, ANY4_EINVAL, ANY4_EALIGN, ANY4_ESHAPE, ANY4_EWORKSPACE, ANY4_ECUDA = 0, -1, -2, -3, -4, -5


class Any4Error(RuntimeError):
    def __init__(self, status: int):
        msg = lib.any4_strerror(status).decode()
        if status == ANY4_ECUDA:
            msg += f" (cudaError {lib.any4_last_cuda_error()})"
        super().__init__(msg)
        self.status = status


def _check(status: int) -> None:
    if status != ANY4_OK:
        raise Any4Error(status)


def _dev(t: torch.Tensor, name: str, itemsize: int, shape=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.element_size() != itemsize:
        raise ValueError(f"{name} must have {itemsize}-byte elements, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


# The current stream's raw handle without building a torch Stream object (the
# binding's per-call cost bounds back-to-back calls of small shapes).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index if device.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(device).cuda_stream


def _stream_of(t: torch.Tensor) -> int:
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


_DECODE_TOKENS = 16   # up to here any4_linear is one kernel


class _Kept:
    """What the binding keeps for a stream. The lock is held from taking the
    workspace to the end of a library call that launches kernels which hand each
    other results through it: ctypes opens the interpreter lock meanwhile, and
    another thread's launches on the stream (every thread starts on the same
    one) may not come between. Reentrant, since a finalizer may make a call of
    its own."""
    __slots__ = ("lock", "workspace")

    def __init__(self):
        self.lock, self.workspace = threading.RLock(), None


_KEPT: dict = {}


def _kept(device: int, stream: int) -> _Kept:
    kept = _KEPT.get((device, stream))
    return kept if kept is not None else _KEPT.setdefault((device, stream), _Kept())


def any4_packed_bytes(n: int, k: int, group: int) -> int:
    return lib.any4_packed_bytes(n, k, group)


def any4_linear_workspace_bytes(m: int, n: int, k: int, group: int) -> int:
    return lib.any4_linear_workspace_bytes(m, n, k, group)


KERNELS = {1: "shared_tables", 2: "register_tables", 3: "prefill_fused", 4: "prefill_gemm",
           5: "shared_tables_direct"}


def any4_linear_kernel(m: int, n: int, k: int, group: int, bits: int = 4) -> str:
    """Name of the kernel any4_linear runs for this shape on the current device."""
    code = lib.any4_linear_kernel(bits, m, n, k, group)
    if code < 0:
        raise Any4Error(code)
    return KERNELS[code]


def any4_linear_grid(m: int, n: int, k: int, group: int, bits: int = 4) -> tuple[int, int]:
    """(thread blocks, blocks per cluster) of the any4_linear launch for this shape."""
    blocks, cluster = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib.any4_linear_grid(bits, m, n, k, group, ctypes.byref(blocks), ctypes.byref(cluster)))
    return blocks.value, cluster.value


def any4_pack(idx_nib: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
              group: int, packed: torch.Tensor | None = None) -> torch.Tensor:
    """Canonical any4 tensors -> device-layout buffer (uint8 tensor)."""
    n, k2 = idx_nib.shape
    k = 2 * k2
    size = any4_packed_bytes(n, k, group)
    if size == 0:
        raise Any4Error(ANY4_ESHAPE)
    dev = idx_nib.device
    if packed is None:
        packed = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(lib.any4_pack(_dev(idx_nib, "idx_nib", 1, (n, k2)), _dev(lut, "lut", 2, (n, 16)),
                         _dev(alpha, "alpha", 2, (n, k // group)),
                         _dev(beta, "beta", 2, (n, k // group)), n, k, group,
                         _dev(packed, "packed", 1), packed.numel(), _stream(dev)))
    return packed


def any4_packed_bytes_bits(bits: int, n: int, k: int, group: int) -> int:
    return lib.any4_packed_bytes_bits(bits, n, k, group)


def any4_pack_bits(bits: int, idx_nib: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
                   beta: torch.Tensor, group: int, packed: torch.Tensor | None = None) -> torch.Tensor:
    """any3 / any2 (bits = 3 / 2; 4 = any4): canonical tensors with indices
    < 2^bits (as nibbles) -> densely packed device-layout buffer."""
    n, k2 = idx_nib.shape
    k = 2 * k2
    size = any4_packed_bytes_bits(bits, n, k, group)
    if size == 0:
        raise Any4Error(ANY4_ESHAPE)
    dev = idx_nib.device
    if packed is None:
        packed = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(lib.any4_pack_bits(bits, _dev(idx_nib, "idx_nib", 1, (n, k2)), _dev(lut, "lut", 2, (n, 16)),
                              _dev(alpha, "alpha", 2, (n, k // group)),
                              _dev(beta, "beta", 2, (n, k // group)), n, k, group,
                              _dev(packed, "packed", 1), packed.numel(), _stream(dev)))
    return packed


def any4_dequant_bits(bits: int, packed: torch.Tensor, n: int, k: int, group: int,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    if out is None:
        out = torch.empty((n, k), dtype=torch.bfloat16, device=packed.device)
    _check(lib.any4_dequant_bits(bits, _dev(packed, "packed", 1), n, k, group, _dev(out, "out", 2, (n, k)),
                                 _stream(packed.device)))
    return out


def any4_linear_bits(bits: int, x: torch.Tensor, packed: torch.Tensor, n: int, k: int, group: int,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    m = x.shape[0]
    if m > _DECODE_TOKENS:
        return _prefill(bits, x, packed, n, k, group, out, workspace)
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = workspace_for(m, n, k, group, x.device, bits)
    _check(lib.any4_linear_bits(bits, _dev(x, "x", 2, (m, k)), _dev(packed, "packed", 1), m, n, k, group,
                                _dev(out, "out", 2, (m, n)), _dev(workspace, "workspace", 1),
                                workspace.numel(), _stream(x.device)))
    return out


def _prefill(bits, x, packed, n, k, group, out, workspace):
    """any4_linear_bits beyond 16 tokens, which may be several kernels."""
    m, x_p = x.shape[0], _dev(x, "x", 2, (x.shape[0], k))
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    out_p, packed_p, stream = _dev(out, "out", 2, (m, n)), _dev(packed, "packed", 1), _stream(x.device)
    with _kept(x.get_device(), stream).lock:
        if workspace is None:
            workspace = workspace_for(m, n, k, group, x.device, bits)
        _check(lib.any4_linear_bits(bits, x_p, packed_p, m, n, k, group, out_p, _dev(workspace, "workspace", 1),
                                    workspace.numel(), stream))
    return out


def any4_dequant(packed: torch.Tensor, n: int, k: int, group: int,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Device-layout buffer -> dequantized W (N x K, bf16)."""
    if out is None:
        out = torch.empty((n, k), dtype=torch.bfloat16, device=packed.device)
    _check(lib.any4_dequant(_dev(packed, "packed", 1), n, k, group, _dev(out, "out", 2, (n, k)),
                            _stream(packed.device)))
    return out


def _refused(bits: int, m: int, n: int, k: int, group: int) -> int:
    """Raises what made a workspace's size 0: the device could not be asked, or
    the call does not take the shape (or its adapters')."""
    code = lib.any4_linear_kernel(bits, m, n, k, group)
    raise Any4Error(code if code == ANY4_ECUDA else ANY4_ESHAPE)


@functools.lru_cache(maxsize=1024)   # a refusal is not kept: it may be a CUDA error that passes
def _linear_need(device: int, *shape: int) -> int:
    """any4_linear_workspace_bytes_bits of a shape (it depends on the device's SM count)."""
    return lib.any4_linear_workspace_bytes_bits(*shape) or _refused(*shape)


@functools.lru_cache(maxsize=1024)
def _lora_need(device: int, *shape: int) -> int:
    return lib.any4_lora_workspace_bytes(*shape) or _refused(*shape[:5])


@functools.lru_cache(maxsize=1024)
def _grad_need(device: int, *shape: int) -> int:
    return lib.any4_lora_grad_workspace_bytes(*shape) or _refused(*shape[:5])


_HEADER_BYTES = lib.any4_lora_header_bytes()
_STATUS_AT = 65536 * 4   # the status word, behind the counters
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)
_WORKSPACES: dict = {}         # of decode calls, a few hundred KB, taken without a lock
_GRAPH_WORKSPACES: dict = {}   # (device, stream): (capture, workspace) of captures under way


def _zeroed(need: int, device: torch.device) -> torch.Tensor:
    """A workspace with the zero header a first call asks for."""
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    ws[:_HEADER_BYTES].zero_()
    return ws


def _graph_workspace(need: int, device: torch.device, key: tuple) -> torch.Tensor:
    """While stream key = (device, stream) is captured: a workspace of the graph's
    own, whose header each replay clears once. Eager calls and other graphs may
    run beside a replay, so it is shared with none of them; the reference kept
    here serves the later calls of the same capture."""
    capture = ctypes.c_uint64(0)
    _check(lib.any4_stream_capture_id(key[1], ctypes.byref(capture)))
    have = _GRAPH_WORKSPACES.get(key)
    if have is None or have[0] != capture.value or have[1].numel() < need:
        have = _GRAPH_WORKSPACES[key] = (capture.value, _zeroed(need, device))
    return have[1]


def _kept_workspace(need: int, device: torch.device, kept: _Kept) -> torch.Tensor:
    """The stream's one workspace for calls of several kernels, which may hold a
    whole dequantized weight; grown on demand. Called with kept.lock held."""
    ws = kept.workspace
    if ws is None or ws.numel() < need:
        ws = kept.workspace = None   # free before the larger one is made
        ws = kept.workspace = _zeroed(need, device)
    return ws


def workspace_for(m: int, n: int, k: int, group: int, device: torch.device, bits: int = 4) -> torch.Tensor:
    """A zero-initialised workspace for this stream, grown on demand and reused
    by later calls on the same stream (calls on one stream never overlap), or,
    while the stream is captured, by the later calls of that capture."""
    key = (device.index if device.index is not None else torch.cuda.current_device(),
           _stream(device))
    need = _linear_need(key[0], bits, m, n, k, group)
    if _capturing():
        return _graph_workspace(need, device, key)
    if _GRAPH_WORKSPACES:
        _GRAPH_WORKSPACES.clear()   # a capture still under way makes itself another
    if m > _DECODE_TOKENS:
        kept = _kept(*key)
        with kept.lock:
            return _kept_workspace(need, device, kept)
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=device)
        _WORKSPACES[key] = ws
    return ws


def any4_linear(x: torch.Tensor, packed: torch.Tensor, n: int, k: int, group: int,
                out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = x . W_hat^T for bf16 x (M x K) -> y (M x N, bf16). M <= 16 runs the
    fused decode kernel, M > 16 the dequantize-then-GEMM prefill path. Any
    number of threads may call it, on one stream or several."""
    m = x.shape[0]
    if m > _DECODE_TOKENS:
        return _prefill(4, x, packed, n, k, group, out, workspace)
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = workspace_for(m, n, k, group, x.device)
    st = lib.any4_linear(_dev(x, "x", 2, (m, k)), _dev(packed, "packed", 1), m, n, k, group,
                         _dev(out, "out", 2, (m, n)), _dev(workspace, "workspace", 1),
                         workspace.numel(), _stream_of(x))
    if st != ANY4_OK:
        raise Any4Error(st)
    return out


def any4_linear_noalloc(x: torch.Tensor, packed: torch.Tensor, n: int, k: int, group: int,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """any4_linear without a workspace, for callers that cannot allocate device
    memory (e.g. an operator inside a runtime that owns all device memory): the
    library's own fixed scratch array is used instead. Calls that may overlap
    on the GPU must be ordered by the caller, since they share that array.
    ``out`` may be passed to avoid the one allocation this Python helper makes."""
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _check(lib.any4_linear_noalloc(_dev(x, "x", 2, (m, k)), _dev(packed, "packed", 1), m, n, k,
                                   group, _dev(out, "out", 2, (m, n)), _stream(x.device)))
    return out


class _DeviceWord:
    """A 32-bit device word exposed through the CUDA array interface."""

    def __init__(self, ptr: int):
        self.__cuda_array_interface__ = {"shape": (1,), "typestr": "<u4", "data": (ptr, False),
                                         "version": 3}


def noalloc_status(device: torch.device | None = None) -> int:
    """The status word of any4_linear_noalloc on ``device`` (0: the last call
    completed normally). Synchronizes that device before reading it."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        ptr = _p()
        _check(lib.any4_noalloc_status_word(ctypes.byref(ptr)))
        torch.cuda.synchronize(dev)
        word = torch.as_tensor(_DeviceWord(ptr.value), device=dev)
        return int(word.view(torch.int32).item()) & 0xFFFFFFFF


def _workspaces_of(device: torch.device) -> list:
    """The workspaces kept for a device's streams."""
    index = device.index if device.index is not None else torch.cuda.current_device()
    found = [ws for key, ws in list(_WORKSPACES.items()) if key[0] == index]
    for key, kept in list(_KEPT.items()):
        if key[0] == index:
            with kept.lock:
                found += [] if kept.workspace is None else [kept.workspace]
    return found


def workspace_status(device: torch.device | None = None) -> int:
    """The status of the calls that were given no workspace, on any stream of
    ``device``: 0 if all completed; bit 0 is set once a bounded wait in a kernel
    gave up, which leaves that call's outputs incomplete and the workspace unfit
    for another call until reset_workspaces. Synchronizes the device. Graphs
    that were captured without a workspace keep their status to themselves."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    torch.cuda.synchronize(dev)
    status = 0
    for ws in _workspaces_of(dev):
        status |= int(ws[_STATUS_AT:_STATUS_AT + 4].view(torch.int32).item()) & 0xFFFFFFFF
    return status


def reset_workspaces(device: torch.device | None = None) -> None:
    """Clears the counters and the status of the workspaces kept for ``device``,
    as before their first use. Synchronizes the device, before and after: no call
    may be made on it meanwhile."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    torch.cuda.synchronize(dev)
    with torch.inference_mode():   # a workspace may have been made in that mode
        for ws in _workspaces_of(dev):
            ws[:_HEADER_BYTES].zero_()
    torch.cuda.synchronize(dev)


def any4_quantize(w: torch.Tensor, ex: torch.Tensor, group: int, bits: int = 4,
                  iters: int = 10):
    """GPU any4 quantizer: bf16 W (N x K) and float64 E|x| (K) -> the canonical
    tensors (idx_nib, lut, alpha, beta) as int16/uint8 device tensors."""
    n, k = w.shape
    dev = w.device
    idx_nib = torch.empty((n, k // 2), dtype=torch.uint8, device=dev)
    lut = torch.empty((n, 16), dtype=torch.int16, device=dev)
    alpha = torch.empty((n, k // group), dtype=torch.int16, device=dev)
    beta = torch.empty((n, k // group), dtype=torch.int16, device=dev)
    if ex.dtype != torch.float64:
        raise ValueError("ex must be float64")
    _check(lib.any4_quantize(_dev(w, "w", 2, (n, k)), _dev(ex, "ex", 8, (k,)), n, k, group, bits,
                             iters, _dev(idx_nib, "idx_nib", 1), _dev(lut, "lut", 2),
                             _dev(alpha, "alpha", 2), _dev(beta, "beta", 2), _stream(dev)))
    return idx_nib, lut, alpha, beta


def _format_code(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def any4_format_lut(fmt) -> list:
    """The 16 bf16 bit patterns of a fixed-table format ("int4", "nf4", "fp4"),
    by code. Host only."""
    buf = (ctypes.c_uint16 * 16)()
    _check(lib.any4_format_lut(_format_code(fmt), ctypes.cast(buf, _p)))
    return [int(v) for v in buf]


def any4_pack_format(fmt, idx_nib: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
                     group: int, packed: torch.Tensor | None = None) -> torch.Tensor:
    """Fixed-table format codes + alpha/beta -> device-layout buffer; the
    format's table goes to every row, so any4_dequant / any4_linear apply."""
    n, k2 = idx_nib.shape
    k = 2 * k2
    size = any4_packed_bytes(n, k, group)
    if size == 0:
        raise Any4Error(ANY4_ESHAPE)
    dev = idx_nib.device
    if packed is None:
        packed = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(lib.any4_pack_format(_format_code(fmt), _dev(idx_nib, "idx_nib", 1, (n, k2)),
                                _dev(alpha, "alpha", 2, (n, k // group)),
                                _dev(beta, "beta", 2, (n, k // group)), n, k, group,
                                _dev(packed, "packed", 1), packed.numel(), _stream(dev)))
    return packed


# ---- low-rank adapters and 8-bit activation checkpoints

def _typed(t: torch.Tensor, name: str, dtypes, device: torch.device, shape) -> int:
    """Pointer of a contiguous CUDA tensor of one of ``dtypes`` on ``device``."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {dtypes[0]}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)   # bf16 values, or their bit patterns
_BYTES = (torch.uint8,)
_INT8, _INT32, _FP32 = (torch.int8,), (torch.int32,), (torch.float32,)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _on_device(name: str):
    """Runs a call with the device of its first tensor, argument ``name``,
    current (the library launches on the current device)."""
    def wrap(call):
        @functools.wraps(call)
        def run(*args, **kwargs):
            t = args[0] if args else kwargs.get(name)
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
                raise ValueError(f"{name} must be a 2-dimensional CUDA tensor")
            if t.get_device() == _current_device():
                return call(*args, **kwargs)
            with torch.cuda.device(t.device):
                return call(*args, **kwargs)
        return run
    return wrap


_packed_need = functools.lru_cache(maxsize=1024)(lambda *shape: lib.any4_packed_bytes_bits(*shape))


def _adapter_workspace(need: int, device: torch.device, stream: int, kept: _Kept) -> torch.Tensor:
    """The stream's workspace, or the graph's that is captured. Called with
    kept.lock held."""
    if _capturing():
        return _graph_workspace(need, device, (device.index, stream))
    if _GRAPH_WORKSPACES:
        _GRAPH_WORKSPACES.clear()
    return _kept_workspace(need, device, kept)


def _adapters(a, b, scale, ids, m: int, n: int, k: int, device: torch.device):
    """Checked adapter arguments: pointers of a, b, scale, ids, then L and R."""
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise ValueError("a must be a tensor of shape (adapters, rank, K)")
    count, rank = a.shape[0], a.shape[1]
    return (_typed(a, "a", _BF16, device, (count, rank, k)), _typed(b, "b", _BF16, device, (count, n, rank)),
            _typed(scale, "scale", _FP32, device, (count,)),
            None if ids is None else _typed(ids, "ids", _INT32, device, (m,)), count, rank)


def _weight(packed, n: int, k: int, group: int, bits: int, device: torch.device) -> int:
    """Pointer of a packed weight that is large enough for its shape."""
    if not isinstance(packed, torch.Tensor):
        raise ValueError("packed must be a CUDA tensor")
    need = _packed_need(bits, n, k, group)
    if need == 0:
        raise Any4Error(ANY4_ESHAPE)
    if packed.numel() < need:
        raise Any4Error(ANY4_EWORKSPACE)
    return _typed(packed, "packed", _BYTES, device, packed.shape)


def any4_lora_workspace_bytes(m: int, n: int, k: int, group: int, adapters: int, rank: int, bits: int = 4) -> int:
    return lib.any4_lora_workspace_bytes(bits, m, n, k, group, adapters, rank)


def any4_lora_grad_workspace_bytes(m: int, n: int, k: int, group: int, adapters: int, rank: int,
                                   bits: int = 4) -> int:
    return lib.any4_lora_grad_workspace_bytes(bits, m, n, k, group, adapters, rank)


@_on_device("x")
def any4_linear_lora(x: torch.Tensor, packed: torch.Tensor, n: int, k: int, group: int, a: torch.Tensor,
                     b: torch.Tensor, scale: torch.Tensor, ids: torch.Tensor | None = None, bits: int = 4,
                     out: torch.Tensor | None = None, u: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = x[t] . W_hat^T + u[t] . B_l^T with u[t] = scale[l] (x[t] . A_l^T)
    and l = ids[t]: the any4 linear layer with one of L low-rank adapters per
    token (a: L x R x K, b: L x N x R bf16, scale: L fp32, ids: M int32; ids
    outside [0, L) have no adapter, None is adapter 0 for every token).
    ``u`` (M x R bf16) is written where given, for any4_linear_lora_grad. Any
    number of threads may make these calls, on one stream or several."""
    m, dev = x.shape[0], x.device
    ad = _adapters(a, b, scale, ids, m, n, k, dev)
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
        out_p = out.data_ptr()
    else:
        out_p = _typed(out, "out", _BF16, dev, (m, n))
    x_p, w_p = _typed(x, "x", _BF16, dev, (m, k)), _weight(packed, n, k, group, bits, dev)
    u_p = None if u is None else _typed(u, "u", _BF16, dev, (m, ad[5]))
    stream = _stream(dev)
    kept = _kept(dev.index, stream)
    with kept.lock:
        if workspace is None:
            workspace = _adapter_workspace(_lora_need(dev.index, bits, m, n, k, group, ad[4], ad[5]), dev, stream,
                                           kept)
        st = lib.any4_linear_lora(bits, x_p, w_p, m, n, k, group, *ad, out_p, u_p,
                                  _typed(workspace, "workspace", _BYTES, dev, workspace.shape), workspace.numel(),
                                  stream)
    if st != ANY4_OK:
        raise Any4Error(st)
    return out


@_on_device("dy")
def any4_linear_lora_grad(dy: torch.Tensor, x, u: torch.Tensor | None, packed: torch.Tensor | None, n: int, k: int,
                          group: int, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor,
                          ids: torch.Tensor | None = None, bits: int = 4,
                          outputs: tuple = ("dx", "da", "db"), dx: torch.Tensor | None = None,
                          da: torch.Tensor | None = None, db: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None) -> tuple:
    """(dx, da, db) of any4_linear_lora for dy (M x N bf16); None for those
    not named in ``outputs``. ``x`` is the forward's bf16 input or the
    (codes, steps) pair any4_act_pack made of it (needed for da), ``u`` what
    the forward wrote (needed for db), ``packed`` the weight (for dx)."""
    m, dev = dy.shape[0], dy.device
    unknown = set(outputs) - {"dx", "da", "db"}
    if unknown or not outputs:
        raise ValueError(f"outputs must name some of dx, da and db, got {tuple(outputs)}")
    ad = _adapters(a, b, scale, ids, m, n, k, dev)
    count, rank = ad[4], ad[5]

    def made(name, t, shape):
        if name not in outputs:
            if t is not None:
                raise ValueError(f"{name} was given but is not among the outputs")
            return None, None
        if t is None:
            t = torch.empty(*shape, dtype=torch.bfloat16, device=dev)
            return t, t.data_ptr()
        return t, _typed(t, name, _BF16, dev, shape)

    dx, dx_p = made("dx", dx, (m, k))
    da, da_p = made("da", da, (count, rank, k))
    db, db_p = made("db", db, (count, n, rank))
    x_p = codes_p = steps_p = None
    x_group = 0
    if da is not None:
        if isinstance(x, (tuple, list)):
            codes, steps = x
            groups = steps.shape[1] if isinstance(steps, torch.Tensor) and steps.dim() == 2 else 0
            if groups < 1 or k % groups:
                raise ValueError("steps must be a tensor of shape (M, K / group)")
            x_group = k // groups
            codes_p = _typed(codes, "codes", _INT8, dev, (m, k))
            steps_p = _typed(steps, "steps", _BF16, dev, (m, groups))
        else:
            x_p = _typed(x, "x", _BF16, dev, (m, k))
    u_p = _typed(u, "u", _BF16, dev, (m, rank)) if db is not None else None
    w_p = _weight(packed, n, k, group, bits, dev) if dx is not None else None
    dy_p = _typed(dy, "dy", _BF16, dev, (m, n))
    stream = _stream(dev)
    kept = _kept(dev.index, stream)
    with kept.lock:
        if workspace is None:
            workspace = _adapter_workspace(_grad_need(dev.index, bits, m, n, k, group, count, rank), dev, stream,
                                           kept)
        _check(lib.any4_linear_lora_grad(
            bits, dy_p, x_p, codes_p, steps_p, x_group, u_p, w_p, m, n, k, group, *ad, dx_p, da_p, db_p,
            _typed(workspace, "workspace", _BYTES, dev, workspace.shape), workspace.numel(), stream))
    return dx, da, db


@_on_device("x")
def any4_act_pack(x: torch.Tensor, group: int, codes: torch.Tensor | None = None,
                  steps: torch.Tensor | None = None) -> tuple:
    """8-bit checkpoint of an activation x (M x K bf16): (codes, steps), one
    int8 per value and one bf16 step per token and ``group`` columns."""
    (m, k), dev = x.shape, x.device
    if group < 1 or k % group:
        raise Any4Error(ANY4_ESHAPE)
    if codes is None:
        codes = torch.empty(m, k, dtype=torch.int8, device=dev)
    if steps is None:
        steps = torch.empty(m, k // group, dtype=torch.bfloat16, device=dev)
    st = lib.any4_act_pack(_typed(x, "x", _BF16, dev, (m, k)), m, k, group, _typed(codes, "codes", _INT8, dev, (m, k)),
                           _typed(steps, "steps", _BF16, dev, (m, k // group)), _stream(dev))
    if st != ANY4_OK:
        raise Any4Error(st)
    return codes, steps


@_on_device("codes")
def any4_act_unpack(codes: torch.Tensor, steps: torch.Tensor, group: int,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """The bf16 values (M x K) an 8-bit checkpoint stands for."""
    (m, k), dev = codes.shape, codes.device
    if group < 1 or k % group:
        raise Any4Error(ANY4_ESHAPE)
    if out is None:
        out = torch.empty(m, k, dtype=torch.bfloat16, device=dev)
    _check(lib.any4_act_unpack(_typed(codes, "codes", _INT8, dev, (m, k)),
                               _typed(steps, "steps", _BF16, dev, (m, k // group)), m, k, group,
                               _typed(out, "out", _BF16, dev, (m, k)), _stream(dev)))
    return out


def any4_strerror(status: int) -> str:
    return lib.any4_strerror(status).decode()
