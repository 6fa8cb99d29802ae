"""Thin binding over libtwell_gb300.so (the C ABI declared in include/twell.h): ctypes for the FFN's calls, the native
module _twell_call for those that a decode step makes many of.

Argument marshalling only: every step of the layer runs in the library's CUDA kernels. PyTorch
provides device memory and the current CUDA stream. The functions carry the C names; each
allocates its outputs with torch when they are not given, passes raw device pointers and the
current stream, and raises TwellError on a non-OK status. There is no fallback: without the
built library every call raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import importlib
import inspect
import math
import os
import threading
from fractions import Fraction
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtwell_gb300.so")

TWELL_OK = 0
TWELL_ERR_UNSUPPORTED = 2
TWELL_BF16 = 0
TWELL_F32 = 1
TWELL_E4M3 = 2
(OP_GATE_PACK, OP_FFN_FUSED_FWD, OP_HYBRID_FWD, OP_HYBRID_BWD, OP_HYBRID_ROUTE, OP_FFN_UNION_FWD, OP_FFN_DECODE,
 OP_FFN_TILE_UNION_FWD, OP_FFN_GATE_UNION_FWD, OP_ADD_RMSNORM_BWD, OP_PAGED_ATTN, OP_LORA_ADD) = range(12)
INT32_MAX = 2 ** 31 - 1  # sizes are 32 bits wide in the C ABI
DECODE_MAX_N = 16  # twell_ffn_decode and twell_w4_matvec take batches of at most this many tokens
STATUS_NAMES = {0: "TWELL_OK", 1: "TWELL_ERR_INVALID", 2: "TWELL_ERR_UNSUPPORTED", 3: "TWELL_ERR_BACKUP_FULL",
                4: "TWELL_ERR_TIMEOUT", 5: "TWELL_ERR_DEVICE_CHECK", 6: "TWELL_ERR_CUDA",
                7: "TWELL_ERR_WORKSPACE", 8: "TWELL_ERR_POOL_EMPTY"}

# Every function the header declares; the CPU tests check that the library exports each one.
EXPORTS = ("twell_packed_vals_bytes", "twell_packed_idx_bytes", "twell_packed_cnt_bytes", "twell_workspace_bytes",
           "twell_gate_pack", "twell_ffn_fused_fwd", "twell_ffn_union_fwd", "twell_hybrid_fwd", "twell_hybrid_bwd", "twell_unpack",
           "twell_pack_from_gate", "twell_hybrid_route_from_gate", "twell_hybrid_route_noalloc",
           "twell_gate_gemm", "twell_gemm_test", "twell_column_activity", "twell_gather_rows",
           "twell_read_status", "twell_status_string", "twell_device_info", "twell_wait_probe",
           "twell_ffn_fused_fwd_f16down", "twell_convert_f16", "twell_ffn_decode", "twell_ffn_tile_union_fwd",
           "twell_count_nonzeros", "twell_convert_f16_transposed", "twell_ffn_gate_union_fwd",
           "twell_add_rmsnorm_fwd", "twell_add_rmsnorm_bwd", "twell_kv_append", "twell_kv_gather",
           "twell_paged_attn_decode", "twell_w4_words_bytes", "twell_w4_scales_bytes", "twell_w4_quantize",
           "twell_w4_matvec", "twell_rope_fwd", "twell_rope_bwd", "twell_kv_plan", "twell_lora_add")


class TwellError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} ({_status_string(code)})")


class _Packed(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int32), ("n_cols", ctypes.c_int32), ("tile", ctypes.c_int32),
                ("cap", ctypes.c_int32), ("dtype", ctypes.c_int), ("vals", ctypes.c_void_p),
                ("idx", ctypes.c_void_p), ("cnt", ctypes.c_void_p)]


class _Hybrid(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int32), ("n_cols", ctypes.c_int32), ("K", ctypes.c_int32),
                ("backup_cap", ctypes.c_int32), ("dtype", ctypes.c_int), ("a", ctypes.c_void_p),
                ("u", ctypes.c_void_p), ("col", ctypes.c_void_p), ("cnt", ctypes.c_void_p),
                ("backup_rows", ctypes.c_void_p), ("n_backup", ctypes.c_void_p), ("A_b", ctypes.c_void_p),
                ("U_b", ctypes.c_void_p), ("l1", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


class _KVCache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64)]


class _RopeHeads(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n_heads", ctypes.c_int32), ("in_batch", ctypes.c_int64),
                ("in_token", ctypes.c_int64), ("in_head", ctypes.c_int64), ("out_batch", ctypes.c_int64),
                ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64)]


class _PagePool(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("ring", ctypes.c_void_p), ("state", ctypes.c_void_p)]


class _Adapters(ctypes.Structure):
    _fields_ = [("n_adapters", ctypes.c_int32), ("rank", ctypes.c_int32), ("k", ctypes.c_int32), ("n", ctypes.c_int32),
                ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ranks", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None
_native = None  # the module _twell_call, once load() has imported it


def _library(path: str = LIB_PATH):
    """The library alone: what the calls that go through ctypes need."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with activation_sparse_ffn_gate_gb300.build.build()")
            lib = ctypes.CDLL(path)
            vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            st = ctypes.c_int
            sig = {
                "twell_packed_vals_bytes": (sz, [i32, i32, i32, ctypes.c_int]),
                "twell_packed_idx_bytes": (sz, [i32, i32, i32]),
                "twell_packed_cnt_bytes": (sz, [i32, i32, i32]),
                "twell_workspace_bytes": (sz, [ctypes.c_int, i32, i32, i32, i32, i32, i32]),
                "twell_gate_pack": (st, [vp, vp, i32, i32, i32, i32, ctypes.c_int, ctypes.POINTER(_Packed), vp, sz,
                                         vp, vp]),
                "twell_ffn_fused_fwd": (st, [vp, vp, vp, ctypes.POINTER(_Packed), i32, i32, i32, ctypes.c_int, vp, vp,
                                             sz, vp, vp]),
                "twell_ffn_union_fwd": (st, [vp, vp, vp, ctypes.POINTER(_Packed), i32, i32, i32, ctypes.c_int, vp, vp,
                                             sz, vp, vp]),
                "twell_ffn_gate_union_fwd": (st, [vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_int,
                                                  ctypes.POINTER(_Packed), vp, vp, sz, vp, vp]),
                "twell_ffn_tile_union_fwd": (st, [vp, vp, vp, ctypes.POINTER(_Packed), i32, i32, i32, vp, vp, sz,
                                                  vp, vp]),
                "twell_wait_probe": (st, [i32, i32, vp, vp]),
                "twell_ffn_fused_fwd_f16down": (st, [vp, vp, vp, ctypes.POINTER(_Packed), i32, i32, i32, vp, vp, sz,
                                                     vp, vp]),
                "twell_convert_f16": (st, [vp, vp, ctypes.c_int64, vp, vp]),
                "twell_convert_f16_transposed": (st, [vp, vp, i32, i32, vp, vp]),
                "twell_ffn_decode": (st, [vp, vp, vp, vp, i32, i32, i32, i32, ctypes.POINTER(_Packed), vp, vp, sz,
                                          vp, vp]),
                "twell_hybrid_fwd": (st, [vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, ctypes.c_int,
                                          ctypes.POINTER(_Hybrid), vp, vp, sz, vp]),
                "twell_hybrid_bwd": (st, [vp, vp, vp, vp, ctypes.POINTER(_Hybrid), vp, i32, i32, i32, ctypes.c_float,
                                          vp, vp, vp, vp, vp, sz, vp]),
                "twell_unpack": (st, [ctypes.POINTER(_Packed), vp, vp, vp]),
                "twell_pack_from_gate": (st, [vp, i32, i32, i32, ctypes.c_int, ctypes.POINTER(_Packed), vp, vp]),
                "twell_hybrid_route_from_gate": (st, [vp, i32, i32, i32, ctypes.c_int, ctypes.POINTER(_Hybrid), vp,
                                                      sz, vp]),
                "twell_hybrid_route_noalloc": (st, [ctypes.POINTER(_Packed), i32, ctypes.POINTER(_Hybrid), vp]),
                "twell_gate_gemm": (st, [vp, vp, i32, i32, i32, vp, vp, vp]),
                "twell_column_activity": (st, [ctypes.POINTER(_Packed), vp, vp, vp]),
                "twell_count_nonzeros": (st, [ctypes.POINTER(_Packed), vp, vp, vp]),
                "twell_gather_rows": (st, [vp, i32, vp, i32, i32, ctypes.c_int, vp, vp, vp]),
                "twell_gemm_test": (st, [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]),
                "twell_add_rmsnorm_fwd": (st, [vp, vp, vp, i32, i32, ctypes.c_float, ctypes.c_int, ctypes.c_int, vp, vp,
                                               vp, vp, i32, vp, vp]),
                "twell_add_rmsnorm_bwd": (st, [vp, vp, vp, vp, vp, i32, i32, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                               vp, vp, vp, sz, vp]),
                "twell_kv_append": (st, [ctypes.POINTER(_KVCache), vp, vp, ctypes.c_int64, ctypes.c_int64, vp, i32, vp,
                                         vp]),
                "twell_kv_gather": (st, [ctypes.POINTER(_KVCache), vp, i32, vp, vp, vp, vp]),
                "twell_paged_attn_decode": (st, [vp, ctypes.c_int64, ctypes.POINTER(_KVCache), vp, vp, i32, i32, i32,
                                                 ctypes.c_float, i32, vp, vp, vp, sz, vp, vp]),
                "twell_w4_words_bytes": (sz, [i32, i32]),
                "twell_w4_scales_bytes": (sz, [i32, i32, i32]),
                "twell_w4_quantize": (st, [vp, i32, i32, i32, vp, vp, vp, vp]),
                "twell_w4_matvec": (st, [vp, vp, vp, i32, i32, i32, i32, vp, vp]),
                "twell_rope_fwd": (st, [ctypes.POINTER(_RopeHeads), ctypes.POINTER(_RopeHeads), vp, ctypes.c_int64, vp,
                                        ctypes.c_float, i32, i32, i32, i32, i32, ctypes.c_int, vp]),
                "twell_rope_bwd": (st, [ctypes.POINTER(_RopeHeads), ctypes.POINTER(_RopeHeads), vp, ctypes.c_int64, vp,
                                        ctypes.c_float, i32, i32, i32, i32, i32, ctypes.c_int, vp]),
                "twell_kv_plan": (st, [ctypes.POINTER(_PagePool), vp, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]),
                "twell_lora_add": (st, [vp, ctypes.c_int64, vp, ctypes.c_int64, ctypes.POINTER(_Adapters), vp, i32, vp,
                                        ctypes.c_int64, vp, sz, vp, vp]),
                "twell_read_status": (st, [vp, vp]),
                "twell_status_string": (ctypes.c_char_p, [ctypes.c_int]),
                "twell_device_info": (st, [ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i32)]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def load(path: str = LIB_PATH):
    """Load the library and the native calls beside it (raises if either has not been built, or not for this torch). A library
    from elsewhere has none beside it: the calls that need them load these, and say if they are missing."""
    global _native
    first = _lib is None
    lib = _library(path)
    if path == LIB_PATH and (first or _native is None):
        try:
            _native = importlib.import_module("._twell_call", __package__)
        except ImportError as e:
            raise RuntimeError(f"the native calls are missing ({e}): build them with "
                               "activation_sparse_ffn_gate_gb300.build.build()") from e
    return lib


def _status_string(code: int) -> str:
    try:
        return _library().twell_status_string(code).decode()
    except Exception:  # the library itself failed to load
        return "?"


def _check(code: int, where: str):
    if code != TWELL_OK:
        raise TwellError(code, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def under_stream(stream):
    """The context in which calls are queued on `stream` and what is allocated belongs to it; None: the current one. Anything
    that has a `cuda_stream` is a stream."""
    return torch.cuda.stream(stream if stream is None or isinstance(stream, torch.cuda.Stream) else
                             torch.cuda.ExternalStream(stream.cuda_stream))


def _on_its_stream(fn):
    """A call that is given a stream runs under it as a whole: the outputs and workspaces that it allocates belong to that
    stream, as the kernels that write them do. On the current one their memory could still be in use by
    that stream's work, and would go back to it while the kernels run."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None:
            return fn(*args, **kwargs)
        with under_stream(stream):
            return fn(*args, **kwargs)

    return call


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """The same for one output, for the calls that a decode step makes many of."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with under_stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return TWELL_BF16
    if dt == torch.float32:
        return TWELL_F32
    raise TypeError(f"unsupported element type {dt}")


_status_bufs = {}


def status_buffer(device=None) -> torch.Tensor:
    """The per-device int32 status word the binding passes as dev_status."""
    dev = torch.device(device if device is not None else torch.cuda.current_device())
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    buf = _status_bufs.get(dev.index)
    if buf is None:
        buf = torch.zeros(1, dtype=torch.int32, device=dev)
        _status_bufs[dev.index] = buf
    return buf


_fused_ws = {}
# Held over a call's launches where the workspace is the stream's: the kernels of one call read what the ones before left
# there, and another thread's on the same stream must not come between them.
_turn = threading.Lock()


def _stream_workspace(cache: dict, n: int, device, stream) -> torch.Tensor:
    """n bytes of the workspace of a device and stream in `cache`, grown on demand: the kernels of one stream run one after
    the other, so calls can share it. A call that is being captured into a graph gets one of its own from the
    graph's memory: the graph may replay on any stream, and after the shared one has been outgrown."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(max(n, 1), dtype=torch.uint8, device=device)
    key = (device.index, _stream(stream).value or 0)
    ws = cache.get(key)
    if ws is None or ws.numel() < n:
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device=device)
        cache[key] = ws
    return ws


@_on_its_stream
def fused_workspace(N: int, d: int, f: int, device=None, stream=None) -> torch.Tensor:
    """The workspace twell_ffn_fused_fwd needs for N rows, d_model d, d_ff f (work counter, split
    plan and the partial rows of split rows), one per device and stream."""
    dev = torch.device(device if device is not None else torch.cuda.current_device())
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return _stream_workspace(_fused_ws, twell_workspace_bytes(OP_FFN_FUSED_FWD, N, d, f, 8), dev, stream)


def twell_read_status(status: Optional[torch.Tensor] = None, stream=None, reset: bool = True) -> int:
    """Synchronise the stream and return the device status code (optionally clearing it)."""
    status = status if status is not None else status_buffer()
    code = _library().twell_read_status(_ptr(status), _stream(stream))
    if reset and code != TWELL_OK:
        status.zero_()
    return code


def twell_wait_probe(arrive: bool, limit_ms: int, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Run the library's bounded mbarrier wait on its own (test export): with arrive=False it runs
    out after limit_ms and records TWELL_ERR_TIMEOUT in the status word."""
    _check(_library().twell_wait_probe(1 if arrive else 0, int(limit_ms), _ptr(status if status is not None else
                                                                             status_buffer()), _stream(stream)),
           "twell_wait_probe")


def check_device_status(where: str = "device", status: Optional[torch.Tensor] = None, stream=None):
    _check(twell_read_status(status, stream), where)


# ------------------------------------------------------------------------------------------ TwELL

@dataclasses.dataclass
class TwELL:
    """A TwELL matrix in device memory (see twell_packed in include/twell.h)."""

    n_rows: int
    n_cols: int
    tile: int
    vals: torch.Tensor  # [n_rows, nt, tile] element type
    idx: torch.Tensor  # [n_rows, nt, tile] uint8
    cnt: torch.Tensor  # [n_rows, nt] int16 storage of uint16 counts

    @property
    def nt(self) -> int:
        return -(-self.n_cols // self.tile)

    @property
    def dtype(self) -> torch.dtype:
        return self.vals.dtype

    @staticmethod
    def empty(n_rows, n_cols, tile, dtype=torch.bfloat16, device=None):
        nt = -(-n_cols // tile)
        device = device or torch.device("cuda", torch.cuda.current_device())
        return TwELL(n_rows, n_cols, tile,
                     torch.empty((n_rows, nt, tile), dtype=dtype, device=device),
                     torch.empty((n_rows, nt, tile), dtype=torch.uint8, device=device),
                     torch.empty((n_rows, nt), dtype=torch.int16, device=device))

    def counts(self) -> torch.Tensor:
        """Counts as non-negative integers (int32)."""
        return self.cnt.to(torch.int32) & 0xFFFF

    def c_struct(self) -> _Packed:
        return _Packed(self.n_rows, self.n_cols, self.tile, self.tile, _dtype_code(self.vals.dtype),
                       self.vals.data_ptr(), self.idx.data_ptr(), self.cnt.data_ptr())


@_on_its_stream
def twell_gate_pack(x: torch.Tensor, Wg_s: torch.Tensor, T: int = 128, out: Optional[TwELL] = None,
                    status: Optional[torch.Tensor] = None, stream=None,
                    vals_dtype: torch.dtype = torch.float32) -> TwELL:
    """Gate GEMM with the ReLU + TwELL pack epilogue: returns the TwELL of ReLU(x Wg_s^T).

    The packed values keep the fp32 accumulator by default (vals_dtype=torch.bfloat16 rounds them)."""
    N, d = x.shape
    f = Wg_s.shape[0]
    out = out if out is not None else TwELL.empty(N, f, T, vals_dtype, x.device)
    s = out.c_struct()
    _check(_library().twell_gate_pack(_ptr(x), _ptr(Wg_s), N, d, f, T, _dtype_code(x.dtype), ctypes.byref(s), None, 0,
                                      _ptr(status if status is not None else status_buffer(x.device)), _stream(stream)),
           "twell_gate_pack")
    return out


@_on_its_stream
def twell_ffn_fused_fwd(x: torch.Tensor, Wu_s: torch.Tensor, Wd_s: torch.Tensor, a: TwELL,
                        y: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                        stream=None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Fused up+down projection over the packed nonzeros: y = (a * (x Wu_s^T)) Wd_s."""
    N, d = x.shape
    f = Wu_s.shape[0]
    y = y if y is not None else torch.empty((N, d), dtype=x.dtype, device=x.device)
    ws = ws if ws is not None else fused_workspace(N, d, f, x.device, stream)
    s = a.c_struct()
    with _turn:
        _check(_library().twell_ffn_fused_fwd(_ptr(x), _ptr(Wu_s), _ptr(Wd_s), ctypes.byref(s), N, d, f,
                                              _dtype_code(x.dtype), _ptr(y), _ptr(ws), ws.numel(),
                                              _ptr(status if status is not None else status_buffer(x.device)),
                                              _stream(stream)),
               "twell_ffn_fused_fwd")
    return y


@_on_its_stream
def twell_convert_f16(src: torch.Tensor, out: Optional[torch.Tensor] = None, status=None,
                      stream=None) -> torch.Tensor:
    """A bf16 tensor converted to fp16 by the library (e.g. Wd_s for twell_ffn_fused_fwd_f16down)."""
    if src.dtype != torch.bfloat16 or not src.is_contiguous():
        raise ValueError("src must be a contiguous bf16 tensor")
    out = out if out is not None else torch.empty(src.shape, dtype=torch.float16, device=src.device)
    _check(_library().twell_convert_f16(_ptr(src), _ptr(out), src.numel(),
                                        _ptr(status if status is not None else status_buffer(src.device)),
                                        _stream(stream)),
           "twell_convert_f16")
    return out


@_on_its_stream
def twell_convert_f16_transposed(src: torch.Tensor, out: Optional[torch.Tensor] = None, status=None,
                                 stream=None) -> torch.Tensor:
    """The transpose of a 2-D bf16 tensor converted to fp16 by the library (e.g. Wd_s [f, d] -> Wd16t_s
    [d, f] for twell_ffn_union_fwd)."""
    if src.dtype != torch.bfloat16 or src.dim() != 2 or not src.is_contiguous():
        raise ValueError("src must be a contiguous 2-D bf16 tensor")
    rows, cols = src.shape
    out = out if out is not None else torch.empty((cols, rows), dtype=torch.float16, device=src.device)
    _check(_library().twell_convert_f16_transposed(_ptr(src), _ptr(out), rows, cols,
                                                   _ptr(status if status is not None else status_buffer(src.device)),
                                                   _stream(stream)),
           "twell_convert_f16_transposed")
    return out


@_on_its_stream
def twell_ffn_fused_fwd_f16down(x: torch.Tensor, Wu_s: torch.Tensor, Wd16_s: torch.Tensor, a: TwELL,
                                y: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                                stream=None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """twell_ffn_fused_fwd with Wd_s given in fp16 (twell_convert_f16) and the down projection in fp16."""
    if Wd16_s.dtype != torch.float16:
        raise ValueError("Wd16_s must be fp16")
    N, d = x.shape
    f = Wu_s.shape[0]
    y = y if y is not None else torch.empty((N, d), dtype=x.dtype, device=x.device)
    ws = ws if ws is not None else fused_workspace(N, d, f, x.device, stream)
    s = a.c_struct()
    with _turn:
        _check(_library().twell_ffn_fused_fwd_f16down(_ptr(x), _ptr(Wu_s), _ptr(Wd16_s), ctypes.byref(s), N, d, f,
                                                      _ptr(y), _ptr(ws), ws.numel(),
                                                      _ptr(status if status is not None else status_buffer(x.device)),
                                                      _stream(stream)),
               "twell_ffn_fused_fwd_f16down")
    return y


class StreamedFFN:
    """The sparse inference FFN over a sequence of batches held in pinned host memory, with each
    batch's copy to the device and its result's copy back overlapped with the neighbouring batches'
    compute: host-to-device copies on one stream, gate + walk (or union path) on a second,
    device-to-host copies on a third, ordered by events, with two device buffers of x and of y
    used in turn. A serving loop so keeps the copy engines and the SMs busy at the same time; the
    kernels and their results are those of ffn_forward."""

    def __init__(self, Wg_s: torch.Tensor, Wu_s: torch.Tensor, Wd_s: torch.Tensor, N: int, T: int = 128,
                 path: str = "walk", vals_dtype: torch.dtype = torch.float32, status: Optional[torch.Tensor] = None,
                 Wd16_s: Optional[torch.Tensor] = None, Wd16t_s: Optional[torch.Tensor] = None):
        dev = Wg_s.device
        f, d = Wg_s.shape
        self.W, self.T, self.path, self.status, self.N, self.d = (Wg_s, Wu_s, Wd_s), T, path, status, N, d
        self.Wd16, self.Wd16t = Wd16_s, Wd16t_s
        self.copy_in, self.compute, self.copy_out = (torch.cuda.Stream(dev) for _ in range(3))
        self.x = [torch.empty((N, d), dtype=Wg_s.dtype, device=dev) for _ in range(2)]
        self.y = [torch.empty((N, d), dtype=Wg_s.dtype, device=dev) for _ in range(2)]
        self.packed = TwELL.empty(N, f, T, vals_dtype, dev)
        self.x_in = [torch.cuda.Event() for _ in range(2)]    # x[b] holds the batch
        self.done = [torch.cuda.Event() for _ in range(2)]    # x[b] read, y[b] written
        self.y_out = [torch.cuda.Event() for _ in range(2)]   # y[b] copied to the host
        self.count = 0

    def submit(self, x_host: torch.Tensor, y_host: torch.Tensor):
        """Queue one batch: x_host [N, d] pinned input, y_host a pinned output of the same shape (valid
        once the copy-out stream has passed it, e.g. after torch.cuda.synchronize())."""
        if tuple(x_host.shape) != (self.N, self.d) or tuple(y_host.shape) != (self.N, self.d):
            raise ValueError("batch shape differs from the pipeline's")
        b, later = self.count % 2, self.count >= 2
        with torch.cuda.stream(self.copy_in):
            if later:
                self.copy_in.wait_event(self.done[b])  # batch count-2 is done reading x[b]
            self.x[b].copy_(x_host, non_blocking=True)
            self.x_in[b].record(self.copy_in)
        with torch.cuda.stream(self.compute):
            self.compute.wait_event(self.x_in[b])
            if later:
                self.compute.wait_event(self.y_out[b])  # y[b] of batch count-2 is on the host
            ffn_forward(self.x[b], *self.W, T=self.T, packed=self.packed, y=self.y[b], status=self.status,
                        stream=self.compute, path=self.path, Wd16_s=self.Wd16, Wd16t_s=self.Wd16t)
            self.done[b].record(self.compute)
        with torch.cuda.stream(self.copy_out):
            self.copy_out.wait_event(self.done[b])
            y_host.copy_(self.y[b], non_blocking=True)
            self.y_out[b].record(self.copy_out)
        self.count += 1


_union_ws = {}


@_on_its_stream
def twell_ffn_union_fwd(x: torch.Tensor, Wu_s: torch.Tensor, Wd16t_s: torch.Tensor, a: TwELL,
                        y: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                        stream=None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The same y as twell_ffn_fused_fwd, as two tensor-core GEMMs over all of d_ff (for dense layers);
    Wd16t_s [d, f] is Wd_s transposed and converted by twell_convert_f16_transposed."""
    N, d = x.shape
    f = Wu_s.shape[0]
    if Wd16t_s.dtype != torch.float16 or tuple(Wd16t_s.shape) != (d, f) or not Wd16t_s.is_contiguous():
        raise ValueError("Wd16t_s must be a contiguous fp16 [d_model, d_ff] tensor "
                         "(twell_convert_f16_transposed of Wd_s)")
    y = y if y is not None else torch.empty((N, d), dtype=x.dtype, device=x.device)
    if ws is None:
        ws = _stream_workspace(_union_ws, twell_workspace_bytes(OP_FFN_UNION_FWD, N, d, f), x.device, stream)
    s = a.c_struct()
    with _turn:
        _check(_library().twell_ffn_union_fwd(_ptr(x), _ptr(Wu_s), _ptr(Wd16t_s), ctypes.byref(s), N, d, f,
                                              _dtype_code(x.dtype), _ptr(y), _ptr(ws), ws.numel(),
                                              _ptr(status if status is not None else status_buffer(x.device)),
                                              _stream(stream)),
               "twell_ffn_union_fwd")
    return y


@_on_its_stream
def twell_ffn_gate_union_fwd(x: torch.Tensor, Wg_s: torch.Tensor, Wu_s: torch.Tensor, Wd16t_s: torch.Tensor,
                             T: int = 128, out: Optional[TwELL] = None, y: Optional[torch.Tensor] = None,
                             status: Optional[torch.Tensor] = None, stream=None, ws: Optional[torch.Tensor] = None,
                             vals_dtype: torch.dtype = torch.float32):
    """twell_gate_pack and twell_ffn_union_fwd with the gate and up projections in one tensor-core
    GEMM: returns (y, the TwELL of ReLU(x Wg_s^T)). T = 64 or 128."""
    N, d = x.shape
    f = Wu_s.shape[0]
    if Wd16t_s.dtype != torch.float16 or tuple(Wd16t_s.shape) != (d, f) or not Wd16t_s.is_contiguous():
        raise ValueError("Wd16t_s must be a contiguous fp16 [d_model, d_ff] tensor "
                         "(twell_convert_f16_transposed of Wd_s)")
    out = out if out is not None else TwELL.empty(N, f, T, vals_dtype, x.device)
    y = y if y is not None else torch.empty((N, d), dtype=x.dtype, device=x.device)
    if ws is None:
        ws = _stream_workspace(_union_ws, twell_workspace_bytes(OP_FFN_GATE_UNION_FWD, N, d, f), x.device, stream)
    s = out.c_struct()
    with _turn:
        _check(_library().twell_ffn_gate_union_fwd(_ptr(x), _ptr(Wg_s), _ptr(Wu_s), _ptr(Wd16t_s), N, d, f, T,
                                                   _dtype_code(x.dtype), ctypes.byref(s), _ptr(y), _ptr(ws), ws.numel(),
                                                   _ptr(status if status is not None else status_buffer(x.device)),
                                                   _stream(stream)),
               "twell_ffn_gate_union_fwd")
    return y, out


_tile_union_ws = {}


@_on_its_stream
def twell_ffn_tile_union_fwd(x: torch.Tensor, Wu_s: torch.Tensor, Wd16_s: torch.Tensor, a: TwELL,
                             y: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                             stream=None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The same y as twell_ffn_fused_fwd, as tensor-core GEMMs over each 128-token tile's union of kept
    units (gathered weight rows); Wd16_s is Wd_s converted by twell_convert_f16."""
    N, d = x.shape
    f = Wu_s.shape[0]
    if Wd16_s.dtype != torch.float16:
        raise ValueError("Wd16_s must be fp16 (twell_convert_f16 of Wd_s)")
    y = y if y is not None else torch.empty((N, d), dtype=x.dtype, device=x.device)
    if ws is None:
        ws = _stream_workspace(_tile_union_ws, twell_workspace_bytes(OP_FFN_TILE_UNION_FWD, N, d, f), x.device, stream)
    s = a.c_struct()
    with _turn:
        _check(_library().twell_ffn_tile_union_fwd(_ptr(x), _ptr(Wu_s), _ptr(Wd16_s), ctypes.byref(s), N, d, f, _ptr(y),
                                                   _ptr(ws), ws.numel(),
                                                   _ptr(status if status is not None else status_buffer(x.device)),
                                                   _stream(stream)),
               "twell_ffn_tile_union_fwd")
    return y


_decode_ws = {}


@_on_its_stream
def twell_ffn_decode(x: torch.Tensor, Wg_s: torch.Tensor, Wu_s: torch.Tensor, Wd_s: torch.Tensor, T: int = 128,
                     packed: Optional[TwELL] = None, y: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None, ws: Optional[torch.Tensor] = None,
                     vals_dtype: torch.dtype = torch.float32):
    """The whole layer for at most DECODE_MAX_N tokens in two launches; returns (y, packed TwELL)."""
    N, d = x.shape
    f = Wg_s.shape[0]
    packed = packed if packed is not None else TwELL.empty(N, f, T, vals_dtype, x.device)
    y = y if y is not None else torch.empty((N, d), dtype=x.dtype, device=x.device)
    if ws is None:
        ws = _stream_workspace(_decode_ws, twell_workspace_bytes(OP_FFN_DECODE, N, d, f, T), x.device, stream)
    s = packed.c_struct()
    with _turn:
        _check(_library().twell_ffn_decode(_ptr(x), _ptr(Wg_s), _ptr(Wu_s), _ptr(Wd_s), N, d, f, T, ctypes.byref(s),
                                           _ptr(y), _ptr(ws), ws.numel(),
                                           _ptr(status if status is not None else status_buffer(x.device)),
                                           _stream(stream)),
               "twell_ffn_decode")
    return y, packed


# Density (kept fraction of d_ff per token) above which the union path beats the walk, measured with
# the whole layer on the 1.5B-like shapes (d_model 2048, d_ff 5632, 8192 tokens, T = 128, L2 flushed; ms):
#   density                               0.1%    0.5%    1%      2%      5%      10%     50%
#   walk (gate + pack, then the walk)     0.188   0.324   0.465   0.782   1.723   3.320   15.27
#   union (gate + up in one GEMM, down)   0.309   0.313   0.313   0.317   0.321   0.340   0.571
#   tile union (gate, then gathered)      0.236   0.378   0.481   0.586   0.688   0.790   1.623
#   dense cuBLAS FFN                      0.365   0.366   0.367   0.366   0.366   0.366   0.369
# The walk's time grows about linearly with the density, so the two cross near 0.45%. On the
# 1.5B-like layer (0.5% kept) the union path is also the faster of the two for every batch of 32 to
# 4096 tokens (us; dense in brackets; up to 128 tokens the union path's products run transposed):
#   tokens      32     64     128    256    512    1024   2048    4096
#   walk        37.7   38.3   46.1   51.5   65.9   89.1   121.2   185.3
#   union       26.7   28.7   32.5   36.4   48.5   65.0   90.0    165.5
#   dense      (31.7) (30.6) (32.7) (36.3) (46.5) (67.3) (111.2) (191.8)
# so batches of up to 4096 tokens switch a little lower, and smaller batches lower still; up to
# UNION_ANY_DENSITY_MAX_N tokens the union path is taken at every density. Uniform layers of those
# shapes at 0.1% / 0.25% kept:
#   64 tokens:  walk 30.8 / 33.0, union 26.8 / 27.3, dense 27.0 / 27.5
#   128 tokens: walk 33.1 / 36.7, union 31.1 / 30.8, dense 29.9 / 29.4
#   256 tokens: walk 34.0 / 43.0, union 34.4 / 34.8, dense 32.8 / 32.9  (cross near 0.1%)
#   512 tokens: walk 38.4 / 51.1, union 48.8 / 48.7, dense 45.6 / 45.3  (cross near 0.22%)
# The gathered tile-union path is never the fastest under these densities; it stays available as path
# "tile_union".
UNION_MIN_DENSITY = 0.0045
UNION_MIN_DENSITY_SMALL_BATCH = 0.004
SMALL_BATCH_MAX_N = 4096
UNION_ANY_DENSITY_MAX_N = 128
# (largest batch, density from which the union path is taken) for batches between those sizes
UNION_MIN_DENSITY_BY_BATCH = ((256, 0.001), (512, 0.002))


def choose_path(n_tokens: int, density: Optional[float]) -> str:
    """The policy of ffn_forward(path="auto"): decode for at most DECODE_MAX_N tokens; the union path
    up to UNION_ANY_DENSITY_MAX_N tokens; above that the walk below a density that grows with the
    batch (UNION_MIN_DENSITY_BY_BATCH, then UNION_MIN_DENSITY_SMALL_BATCH up to SMALL_BATCH_MAX_N
    tokens, then UNION_MIN_DENSITY) or without a density estimate, the union path (gate and up
    projection in one GEMM, down GEMM over all of d_ff) from it on."""
    if n_tokens <= DECODE_MAX_N:
        return "decode"
    if n_tokens <= UNION_ANY_DENSITY_MAX_N:
        return "union"
    limit = UNION_MIN_DENSITY_SMALL_BATCH if n_tokens <= SMALL_BATCH_MAX_N else UNION_MIN_DENSITY
    for max_n, d in UNION_MIN_DENSITY_BY_BATCH:
        if n_tokens <= max_n:
            limit = d
            break
    if density is None or density < limit:
        return "walk"
    return "union"


def ffn_forward(x, Wg_s, Wu_s, Wd_s, T: int = 128, packed: Optional[TwELL] = None, y=None, status=None, stream=None,
                vals_dtype: torch.dtype = torch.float32, path: str = "walk", Wd16_s: Optional[torch.Tensor] = None,
                density: Optional[float] = None, Wd16t_s: Optional[torch.Tensor] = None):
    """The sparse inference FFN: twell_gate_pack, then twell_ffn_fused_fwd (path "walk"),
    twell_ffn_union_fwd (path "union", with Wd16t_s = twell_convert_f16_transposed(Wd_s); for
    T = 64 or 128 as twell_ffn_gate_union_fwd, gate and up projection in one GEMM) or
    twell_ffn_tile_union_fwd (path "tile_union", with Wd16_s = twell_convert_f16(Wd_s)); path
    "decode" runs twell_ffn_decode (at most DECODE_MAX_N tokens). Path "auto" follows choose_path
    with `density`, the kept fraction of the previous batch (twell_count_nonzeros / (N * d_ff));
    without Wd16t_s it stays on the walk."""
    if path == "auto":
        path = choose_path(x.shape[0], density)
        if path == "union" and Wd16t_s is None:
            path = "walk"
        if path == "decode":
            try:
                return twell_ffn_decode(x, Wg_s, Wu_s, Wd_s, T, packed=packed, y=y, status=status, stream=stream,
                                        vals_dtype=vals_dtype)[0]
            except TwellError as e:
                if e.code != TWELL_ERR_UNSUPPORTED:
                    raise
            path = "walk"
    if path == "decode":
        return twell_ffn_decode(x, Wg_s, Wu_s, Wd_s, T, packed=packed, y=y, status=status, stream=stream,
                                vals_dtype=vals_dtype)[0]
    if path == "union" and Wd16t_s is None:
        raise ValueError('path "union" needs Wd16t_s (twell_convert_f16_transposed(Wd_s))')
    if path == "union" and T in (64, 128):
        return twell_ffn_gate_union_fwd(x, Wg_s, Wu_s, Wd16t_s, T, out=packed, y=y, status=status, stream=stream,
                                        vals_dtype=vals_dtype)[0]
    a = twell_gate_pack(x, Wg_s, T, out=packed, status=status, stream=stream, vals_dtype=vals_dtype)
    if path == "union":
        return twell_ffn_union_fwd(x, Wu_s, Wd16t_s, a, y=y, status=status, stream=stream)
    if path == "tile_union":
        if Wd16_s is None:
            raise ValueError('path "tile_union" needs Wd16_s (twell_convert_f16(Wd_s))')
        return twell_ffn_tile_union_fwd(x, Wu_s, Wd16_s, a, y=y, status=status, stream=stream)
    if path != "walk":
        raise ValueError(f"unknown path {path!r}")
    return twell_ffn_fused_fwd(x, Wu_s, Wd_s, a, y=y, status=status, stream=stream)


@_on_its_stream
def twell_unpack(a: TwELL, out: Optional[torch.Tensor] = None, status=None, stream=None) -> torch.Tensor:
    out = out if out is not None else torch.empty((a.n_rows, a.n_cols), dtype=a.dtype, device=a.vals.device)
    s = a.c_struct()
    _check(_library().twell_unpack(ctypes.byref(s), _ptr(out),
                                   _ptr(status if status is not None else status_buffer(out.device)), _stream(stream)),
           "twell_unpack")
    return out


@_on_its_stream
def twell_column_activity(a: TwELL, counts: Optional[torch.Tensor] = None, status=None, stream=None) -> torch.Tensor:
    """Per-column count of the rows of `a` that keep the column (added to `counts`, zeros if None)."""
    counts = counts if counts is not None else torch.zeros(a.n_cols, dtype=torch.int32, device=a.vals.device)
    s = a.c_struct()
    _check(_library().twell_column_activity(ctypes.byref(s), _ptr(counts),
                                            _ptr(status if status is not None else status_buffer(counts.device)),
                                            _stream(stream)),
           "twell_column_activity")
    return counts


@_on_its_stream
def twell_count_nonzeros(a: TwELL, total: Optional[torch.Tensor] = None, status=None, stream=None) -> torch.Tensor:
    """Device int64 [1]: the number of kept entries of `a` (added to `total`, zeros if None)."""
    total = total if total is not None else torch.zeros(1, dtype=torch.int64, device=a.vals.device)
    s = a.c_struct()
    _check(_library().twell_count_nonzeros(ctypes.byref(s), _ptr(total),
                                           _ptr(status if status is not None else status_buffer(total.device)),
                                           _stream(stream)),
           "twell_count_nonzeros")
    return total


@_on_its_stream
def twell_gather_rows(src: torch.Tensor, rows: torch.Tensor, out: Optional[torch.Tensor] = None, status=None,
                      stream=None) -> torch.Tensor:
    """out[i] = src[rows[i]] (rows: int32 device tensor)."""
    n_src, d = src.shape
    n = rows.numel()
    out = out if out is not None else torch.empty((n, d), dtype=src.dtype, device=src.device)
    _check(_library().twell_gather_rows(_ptr(src), n_src, _ptr(rows), n, d, _dtype_code(src.dtype), _ptr(out),
                                        _ptr(status if status is not None else status_buffer(src.device)),
                                        _stream(stream)),
           "twell_gather_rows")
    return out


def live_columns(counts: torch.Tensor) -> torch.Tensor:
    """Ascending int32 indices (on the counts' device) of the columns that fired at least once;
    computed on the host, once per model."""
    import numpy as np
    live = np.flatnonzero(counts.cpu().numpy() > 0).astype(np.int32)
    return torch.from_numpy(live).to(counts.device)


def compact_weights(Wg_s, Wu_s, Wd_s, live: torch.Tensor, status=None, stream=None):
    """The rows of Wg_s, Wu_s, Wd_s of the live hidden units, in the order of `live`."""
    return tuple(twell_gather_rows(W, live, status=status, stream=stream) for W in (Wg_s, Wu_s, Wd_s))


@_on_its_stream
def twell_pack_from_gate(G: torch.Tensor, T: int = 128, out: Optional[TwELL] = None, status=None,
                         stream=None) -> TwELL:
    N, f = G.shape
    out = out if out is not None else TwELL.empty(N, f, T, G.dtype, G.device)
    s = out.c_struct()
    _check(_library().twell_pack_from_gate(_ptr(G), N, f, T, _dtype_code(G.dtype), ctypes.byref(s),
                                           _ptr(status if status is not None else status_buffer(G.device)),
                                           _stream(stream)),
           "twell_pack_from_gate")
    return out


@_on_its_stream
def twell_gate_gemm(x: torch.Tensor, Wg_s: torch.Tensor, out: Optional[torch.Tensor] = None, status=None,
                    stream=None) -> torch.Tensor:
    N, d = x.shape
    f = Wg_s.shape[0]
    out = out if out is not None else torch.empty((N, f), dtype=torch.float32, device=x.device)
    _check(_library().twell_gate_gemm(_ptr(x), _ptr(Wg_s), N, d, f, _ptr(out),
                                      _ptr(status if status is not None else status_buffer(x.device)), _stream(stream)),
           "twell_gate_gemm")
    return out


def twell_workspace_bytes(op: int, N: int, d: int, f: int, tile: int = 128, K: int = 0, backup_cap: int = 0) -> int:
    return int(_library().twell_workspace_bytes(op, N, d, f, tile, K, backup_cap))


def twell_device_info():
    sm, ma, mi = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(_library().twell_device_info(ctypes.byref(sm), ctypes.byref(ma), ctypes.byref(mi)), "twell_device_info")
    return sm.value, ma.value, mi.value


@_on_its_stream
def twell_gemm_test(A: torch.Tensor, B: torch.Tensor, a_mn: bool, b_mn: bool, status=None, stream=None) -> torch.Tensor:
    """C = A_logical @ B_logical (fp32) where A is [M,K] (or [K,M] if a_mn) and B is [N,K] (or [K,N] if b_mn)."""
    M = A.shape[1] if a_mn else A.shape[0]
    K = A.shape[0] if a_mn else A.shape[1]
    N = B.shape[1] if b_mn else B.shape[0]
    C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _check(_library().twell_gemm_test(_ptr(A), _ptr(B), M, N, K, int(a_mn), int(b_mn), _ptr(C),
                                      _ptr(status if status is not None else status_buffer(A.device)), _stream(stream)),
           "twell_gemm_test")
    return C


# ------------------------------------------------------------------------------------------ hybrid format

@dataclasses.dataclass
class Hybrid:
    """A hybrid sparse-block / dense-backup context in device memory (twell_hybrid in include/twell.h)."""

    n_rows: int
    n_cols: int
    K: int
    backup_cap: int
    a: torch.Tensor  # [N, K] fp32
    u: torch.Tensor  # [N, K] fp32
    col: torch.Tensor  # [N, K] int16 storage of uint16 columns
    cnt: torch.Tensor  # [N] int16 storage of uint16 counts (0xFFFF = backup row)
    backup_rows: torch.Tensor  # [cap] int32
    n_backup: torch.Tensor  # [1] int32
    A_b: torch.Tensor  # [cap, f] fp32
    U_b: torch.Tensor  # [cap, f] fp32
    l1: torch.Tensor  # [1] fp32
    status: torch.Tensor  # [1] int32

    @staticmethod
    def empty(n_rows, n_cols, K, backup_cap, device=None):
        device = device or torch.device("cuda", torch.cuda.current_device())
        cap = max(int(backup_cap), 0)
        z = dict(device=device)
        return Hybrid(n_rows, n_cols, K, cap,
                      torch.empty((n_rows, K), dtype=torch.float32, **z),
                      torch.empty((n_rows, K), dtype=torch.float32, **z),
                      torch.empty((n_rows, K), dtype=torch.int16, **z),
                      torch.empty((n_rows,), dtype=torch.int16, **z),
                      torch.empty((max(cap, 1),), dtype=torch.int32, **z),
                      torch.zeros((1,), dtype=torch.int32, **z),
                      torch.empty((max(cap, 1), n_cols), dtype=torch.float32, **z),
                      torch.empty((max(cap, 1), n_cols), dtype=torch.float32, **z),
                      torch.zeros((1,), dtype=torch.float32, **z),
                      torch.zeros((1,), dtype=torch.int32, **z))

    def counts(self) -> torch.Tensor:
        return self.cnt.to(torch.int32) & 0xFFFF

    def cols(self) -> torch.Tensor:
        return self.col.to(torch.int32) & 0xFFFF

    def c_struct(self) -> _Hybrid:
        def ptr(t):
            return t.data_ptr() if t is not None else None
        return _Hybrid(self.n_rows, self.n_cols, self.K, self.backup_cap, TWELL_BF16, ptr(self.a), ptr(self.u),
                       ptr(self.col), ptr(self.cnt), ptr(self.backup_rows), ptr(self.n_backup), ptr(self.A_b),
                       ptr(self.U_b), ptr(self.l1), ptr(self.status))


def _workspace(op, N, d, f, K, cap, device, ws=None):
    nbytes = twell_workspace_bytes(op, N, d, f, 0, K, cap)
    if ws is not None and ws.numel() >= nbytes:
        return ws
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


@_on_its_stream
def twell_hybrid_route_from_gate(G: torch.Tensor, K: int, backup_cap: int, ctx: Optional[Hybrid] = None, ws=None,
                                 stream=None) -> Hybrid:
    N, f = G.shape
    ctx = ctx if ctx is not None else Hybrid.empty(N, f, K, backup_cap, G.device)
    ws = _workspace(OP_HYBRID_ROUTE, N, 8, f, K, ctx.backup_cap, G.device, ws)
    s = ctx.c_struct()
    _check(_library().twell_hybrid_route_from_gate(_ptr(G), N, f, K, TWELL_BF16, ctypes.byref(s), _ptr(ws), ws.numel(),
                                                   _stream(stream)), "twell_hybrid_route_from_gate")
    return ctx


@_on_its_stream
def twell_hybrid_fwd(x, Wg_s, Wu_s, Wd_s, K: int, backup_cap: int, l1_coef: float = 2e-5,
                     ctx: Optional[Hybrid] = None, y=None, ws=None, stream=None):
    """Hybrid-format training forward: returns (y, ctx)."""
    N, d = x.shape
    f = Wg_s.shape[0]
    ctx = ctx if ctx is not None else Hybrid.empty(N, f, K, backup_cap, x.device)
    y = y if y is not None else torch.empty((N, d), dtype=x.dtype, device=x.device)
    ws = _workspace(OP_HYBRID_FWD, N, d, f, K, ctx.backup_cap, x.device, ws)
    s = ctx.c_struct()
    _check(_library().twell_hybrid_fwd(_ptr(x), _ptr(Wg_s), _ptr(Wu_s), _ptr(Wd_s), N, d, f, K, ctypes.c_float(l1_coef),
                                       TWELL_BF16, ctypes.byref(s), _ptr(y), _ptr(ws), ws.numel(), _stream(stream)),
           "twell_hybrid_fwd")
    return y, ctx


@_on_its_stream
def twell_hybrid_bwd(x, Wg_s, Wu_s, Wd_s, ctx: Hybrid, dy, l1_coef: float = 2e-5, dx=None, dWg_s=None, dWu_s=None,
                     dWd_s=None, ws=None, stream=None):
    """Hybrid-format training backward: returns (dx, dWg_s, dWu_s, dWd_s), all fp32."""
    N, d = x.shape
    f = Wg_s.shape[0]
    dx = dx if dx is not None else torch.empty((N, d), dtype=torch.float32, device=x.device)
    dWg_s = dWg_s if dWg_s is not None else torch.empty((f, d), dtype=torch.float32, device=x.device)
    dWu_s = dWu_s if dWu_s is not None else torch.empty((f, d), dtype=torch.float32, device=x.device)
    dWd_s = dWd_s if dWd_s is not None else torch.empty((f, d), dtype=torch.float32, device=x.device)
    ws = _workspace(OP_HYBRID_BWD, N, d, f, ctx.K, ctx.backup_cap, x.device, ws)
    s = ctx.c_struct()
    _check(_library().twell_hybrid_bwd(_ptr(x), _ptr(Wg_s), _ptr(Wu_s), _ptr(Wd_s), ctypes.byref(s), _ptr(dy), N, d, f,
                                       ctypes.c_float(l1_coef), _ptr(dx), _ptr(dWg_s), _ptr(dWu_s), _ptr(dWd_s), _ptr(ws),
                                       ws.numel(), _stream(stream)), "twell_hybrid_bwd")
    return dx, dWg_s, dWu_s, dWd_s


def twell_hybrid_route_noalloc(a: TwELL, K: int, ctx: Hybrid, stream=None) -> Hybrid:
    """Route a packed TwELL (fp32 values, tile 128) into `ctx` with no workspace and no allocation
    in the library (see twell_hybrid_route_noalloc in include/twell.h for who needs this)."""
    sa, sc = a.c_struct(), ctx.c_struct()
    _check(_library().twell_hybrid_route_noalloc(ctypes.byref(sa), K, ctypes.byref(sc), _stream(stream)),
           "twell_hybrid_route_noalloc")
    return ctx


# ------------------------------------------------------------------- the decoder layer around the FFN

# A decode step makes many calls whose kernels take a few microseconds, so their tensors are checked and their
# pointers, stream and workspace taken by the native module _twell_call (csrc/twell_call.cpp): a tensor of the wrong
# shape, type, layout or device raises ValueError there.

def _calls():
    """The native module (load() imports it beside the library)."""
    if _native is None:
        load()
    return _native


def _status(status, index: int) -> torch.Tensor:
    if status is None:
        if index < 0:
            raise ValueError("the call's tensors must be on a GPU")
        status = _status_bufs.get(index)
        if status is None:
            status = status_buffer(torch.device("cuda", index))
    return status


@dataclasses.dataclass
class Rows8:
    """Rows in e4m3 with scales: values[i, j] * scale[i, j // group] (group 0: one scale a row)."""

    values: torch.Tensor  # [N, d] float8_e4m3fn
    scale: torch.Tensor  # [N, groups] fp32
    group: int

    @staticmethod
    def empty(n_rows: int, d: int, group: int = 0, device=None):
        device = device or torch.device("cuda", torch.cuda.current_device())
        ng = -(-d // group) if group else 1
        return Rows8(torch.empty((n_rows, d), dtype=torch.float8_e4m3fn, device=device),
                     torch.empty((n_rows, ng), dtype=torch.float32, device=device), group)


def twell_add_rmsnorm_fwd(x: torch.Tensor, w: torch.Tensor, res: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          y: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                          rstd: Optional[torch.Tensor] = None, training: bool = False, stream=None):
    """The residual addition and RMS norm: h = x + res, y = h * rstd * w with rstd = 1/sqrt(mean(h^2) + eps).

    x [N, d] and w [d] in one type (bf16 or fp32), res in that type or fp32. Returns (y, h, rstd): h is None
    without res (it is x then), rstd None unless training is set or a buffer given. h may be res itself
    and y may be x: the call then works in place."""
    if y is None:
        y = _empty(x.shape, x.dtype, x.device, stream)
    if h is None and res is not None:
        h = _empty(res.shape, res.dtype, res.device, stream)
    if rstd is None and training:
        rstd = _empty(x.shape[:1], torch.float32, x.device, stream)
    code = (_native or _calls()).add_rmsnorm_fwd(x, w, res, eps, h, y, None, None, 0, rstd,
                                                 None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_add_rmsnorm_fwd")
    return y, h, rstd


def twell_add_rmsnorm_fwd_q8(x: torch.Tensor, w: torch.Tensor, res: Optional[torch.Tensor] = None, eps: float = 1e-6,
                             group: int = 0, out: Optional[Rows8] = None, y: Optional[torch.Tensor] = None,
                             h: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                             training: bool = False, stream=None):
    """twell_add_rmsnorm_fwd with y in e4m3, one scale a row (group 0) or per 128 columns (group 128):
    returns (Rows8, h, rstd). y is written in x's type as well when a buffer for it is given."""
    if out is None:
        ng = -(-x.shape[-1] // group) if group else 1
        out = Rows8(_empty(x.shape, torch.float8_e4m3fn, x.device, stream),
                    _empty((x.shape[0], ng), torch.float32, x.device, stream), group)
    if h is None and res is not None:
        h = _empty(res.shape, res.dtype, res.device, stream)
    if rstd is None and training:
        rstd = _empty(x.shape[:1], torch.float32, x.device, stream)
    code = (_native or _calls()).add_rmsnorm_fwd(x, w, res, eps, h, y, out.values, out.scale, out.group, rstd,
                                                 None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_add_rmsnorm_fwd")
    return out, h, rstd


def twell_add_rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor,
                          dh: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                          dw: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Gradients of the call above from its h (x where it had no res) and rstd: returns (dx, dw), dx the
    gradient of x and of res alike, dw fp32. dy, dh (the gradient that reaches h from the residual
    stream, or None) and dx share a type, bf16 or fp32. ws as in twell_paged_attn_decode."""
    if dx is None:
        dx = _empty(dy.shape, dy.dtype, dy.device, stream)
    if dw is None:
        dw = _empty(h.shape[1:], torch.float32, h.device, stream)
    code = (_native or _calls()).add_rmsnorm_bwd(dy, h, w, rstd, dh, dx, dw, ws,
                                                 None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_add_rmsnorm_bwd")
    return dx, dw


def _strides(t: torch.Tensor) -> tuple:
    """A tensor's strides, with that of a contiguous one for an axis of size one, which addresses nothing."""
    out, dense = [], 1
    for size, stride in zip(reversed(t.shape), reversed(t.stride())):
        out.append(dense if size == 1 else stride)
        dense *= size
    return tuple(reversed(out))


class KVCache:
    """A paged key-value cache in device memory (twell_kv_cache in include/twell.h): k and v
    [n_pages, n_kv_heads, page_size, head_dim] in bf16, or in float8_e4m3fn with fp32 scales
    [n_pages, n_kv_heads, page_size]. Any strides with head_dim contiguous will do (a [n_pages, page_size,
    n_kv_heads, head_dim] buffer permuted, halves of one buffer), the same for k and v. Token slot
    s is offset s % page_size of page s // page_size."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device or not k.is_cuda:
            raise ValueError("k and v must be device tensors of one shape [n_pages, n_kv_heads, page_size, head_dim] and type")
        stride = _strides(k)
        if stride != _strides(v) or (k.numel() > 0 and stride[3] != 1):
            raise ValueError("k and v must have the same strides, head_dim contiguous")
        if max(k.shape) > INT32_MAX:
            raise ValueError(f"the cache's sizes must fit 32 bits, not {tuple(k.shape)}")
        q8 = k.dtype == torch.float8_e4m3fn
        if not q8 and k.dtype != torch.bfloat16:
            raise TypeError(f"unsupported cache type {k.dtype}")
        sp = sh = 0
        if q8:
            for s in (k_scale, v_scale):
                if s is None or s.shape != k.shape[:3] or s.dtype != torch.float32 or s.device != k.device:
                    raise ValueError("an e4m3 cache needs fp32 scales [n_pages, n_kv_heads, page_size]")
            sp, sh, st = _strides(k_scale)
            if (sp, sh, st) != _strides(v_scale) or st != 1:
                raise ValueError("the scales must have the same strides, a page's tokens adjacent")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.dtype, self.device, self.index = k.dtype, k.device, k.get_device()
        self._c = _KVCache(self.n_pages, self.page_size, self.n_kv_heads, self.head_dim,
                           TWELL_E4M3 if q8 else TWELL_BF16, k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if q8 else None,
                           v_scale.data_ptr() if q8 else None,
                           *stride[:3], sp, sh)
        self._at = ctypes.addressof(self._c)

    @staticmethod
    def empty(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, dtype: torch.dtype = torch.bfloat16,
              device=None):
        """An empty cache; its slots hold nothing until they are written (an e4m3 cache's scales are zero)."""
        device = device or torch.device("cuda", torch.cuda.current_device())
        k, v = (torch.empty((n_pages, n_kv_heads, page_size, head_dim), dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return KVCache(k, v)
        return KVCache(k, v, *(torch.zeros((n_pages, n_kv_heads, page_size), dtype=torch.float32, device=device)
                               for _ in range(2)))


def twell_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, status=None,
                    stream=None) -> None:
    """Write n tokens' keys and values (bf16 [n, n_kv_heads, head_dim]; any token stride, heads
    contiguous) to their slots (int32 [n], -1 = skip; no slot twice), quantised where the cache is in e4m3."""
    dev = cache.index
    code = (_native or _calls()).kv_append(cache._at, dev, k, v, slots, _status(status, dev),
                                           None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_kv_append")


def twell_kv_gather(cache: KVCache, slots: torch.Tensor, k_out: Optional[torch.Tensor] = None,
                    v_out: Optional[torch.Tensor] = None, status=None, stream=None):
    """Read slots back: (k, v), bf16 [n, n_kv_heads, head_dim]; zeros for slot -1."""
    dev = cache.index
    if k_out is None:
        k_out = _empty((slots.numel(), cache.n_kv_heads, cache.head_dim), torch.bfloat16, cache.device, stream)
    if v_out is None:
        v_out = _empty((slots.numel(), cache.n_kv_heads, cache.head_dim), torch.bfloat16, cache.device, stream)
    code = (_native or _calls()).kv_gather(cache._at, dev, slots, k_out, v_out, _status(status, dev),
                                           None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_kv_gather")
    return k_out, v_out


def twell_paged_attn_decode(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
                            scale: Optional[float] = None, window: int = 0, out: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, status=None,
                            stream=None):
    """Attention of one new token per sequence over the paged cache: returns (out, lse).

    q bf16 [B, n_q_heads, head_dim] (any sequence stride, heads contiguous); page_table int32
    [B, max_pages]; seq_lens int32 [B] (the new token's own slot counted, if it is to be seen); scale
    1/sqrt(head_dim) unless given; window > 0 keeps the last `window` tokens. out bf16, written; lse fp32
    [B, n_q_heads] (natural logarithm of the sum of exponentials) is written when a buffer is given. A
    sequence of length 0 gives zeros and -inf. ws: the caller's workspace; without one the calls of a stream share
    theirs, and a call that is captured into a graph has its own in the graph's memory."""
    dev = cache.index
    if out is None:
        out = _empty(q.shape, torch.bfloat16, cache.device, stream)
    if scale is None:
        scale = cache.head_dim ** -0.5
    code = (_native or _calls()).paged_attn_decode(q, cache._at, dev, page_table, seq_lens, scale, window, out, lse, ws,
                                                   _status(status, dev), None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_paged_attn_decode")
    return out, lse


@dataclasses.dataclass
class W4Weights:
    """4-bit weights [n, k] with a bf16 scale per `group` columns, in the layout of include/twell.h."""

    words: torch.Tensor  # int32 [ceil(n/16), ceil(k/128), 8, 4, 2, 4]
    scales: torch.Tensor  # bf16 [ceil(n/16), ceil(k/128), 8, 2, 128/group]
    n: int
    k: int
    group: int

    def __post_init__(self):
        if self.group not in (32, 64, 128) or self.n <= 0 or self.k <= 0 or self.k % 32 or self.k % self.group:
            raise ValueError("W4Weights: group 32, 64 or 128, k a multiple of 32 and of group")
        tiles = (-(-self.n // 16), -(-self.k // 128))
        for t, shape, dtype, what in ((self.words, tiles + (8, 4, 2, 4), torch.int32, "words"),
                                      (self.scales, tiles + (8, 2, 128 // self.group), torch.bfloat16, "scales")):
            if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.device != self.words.device:
                raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {shape} on one device")

    def dequantize(self) -> torch.Tensor:
        """The fp32 weights [n, k] that the codes stand for (a check, not a fast path)."""
        nt, kt = self.words.shape[:2]
        shift = torch.tensor([[0, 16], [4, 20], [8, 24], [12, 28]], device=self.words.device, dtype=torch.int32)
        c = (self.words[..., None, None] >> shift) & 15
        c = c.permute(0, 4, 2, 1, 5, 3, 6, 7).reshape(nt * 16, kt * 128)
        s = self.scales.permute(0, 3, 2, 1, 4).reshape(nt * 16, -1).float().repeat_interleave(self.group, dim=1)
        return ((c - 8).float() * s)[:self.n, :self.k]


@_on_its_stream
def twell_w4_quantize(W: torch.Tensor, group: int = 128, status=None, stream=None) -> W4Weights:
    """bf16 weights [n, k] quantised to 4 bits with a scale per `group` columns, laid out for
    twell_w4_matvec (once per weight)."""
    if W.dim() != 2 or W.dtype != torch.bfloat16 or not W.is_contiguous() or not W.is_cuda:
        raise ValueError("W must be a contiguous 2-D bf16 tensor on the GPU")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    n, k = W.shape
    if max(n, k) > INT32_MAX:
        raise ValueError(f"the weights' sizes must fit 32 bits, not {n} x {k}")
    nt, kt = -(-n // 16), -(-k // 128)
    words = torch.empty((nt, kt, 8, 4, 2, 4), dtype=torch.int32, device=W.device)
    scales = torch.empty((nt, kt, 8, 2, 128 // group), dtype=torch.bfloat16, device=W.device)
    out = W4Weights(words, scales, n, k, group)
    with torch.cuda.device(W.device):
        _check(_library().twell_w4_quantize(_ptr(W), n, k, group, _ptr(words), _ptr(scales),
                                            _ptr(_status(status, W.get_device())), _stream(stream)),
               "twell_w4_quantize")
    return out


def twell_w4_matvec(x: torch.Tensor, W: W4Weights, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = x W^T (bf16) for at most DECODE_MAX_N tokens and 4-bit weights."""
    if y is None:
        y = _empty((x.shape[0], W.n), torch.bfloat16, x.device, stream)
    code = (_native or _calls()).w4_matvec(x, W.words, W.scales, W.n, W.k, W.group, y,
                                           None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_w4_matvec")
    return y


# What a served step needs beside the layer's own calls: the plan of its tokens, their rotation, and adapters.

# 1 / 2 pi times 2^160, to the last bit but one: pi to 2^-166
_TURN = int(2 ** 159 / Fraction("3.14159265358979323846264338327950288419716939937510"))


def scaled_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original: int = 0,
                       low: Optional[float] = None, high: Optional[float] = None):
    """(frequencies, factor) for Rotary: radians a position of each of rot_dim / 2 pairs, f_i = base^(-2i / rot_dim), changed
    for contexts `factor` times as long as the `original` length a model was trained at:
    "none"; "linear": f / factor; "base": base times factor^(rot_dim / (rot_dim - 2)), so that the first pair stays and the
    last becomes f / factor; "bands": by the number of turns n_i = original f_i / 2 pi, f where n >= high (4), f / factor
    where n <= low (1), between them (1 - s) f / factor + s f with s = (n - low) / (high - low); "ramp": by the index of the
    pair, i(n) = rot_dim ln(original / (2 pi n)) / (2 ln base), f up to floor(i(high)) (high 32 turns), f / factor from
    ceil(i(low)) (1 turn) on, a straight line between them, and turned values times 0.1 ln(factor) + 1."""
    if rot_dim < 2 or rot_dim % 2 or not base > 1 or not factor >= 1:
        raise ValueError("rot_dim must be even, base above 1 and factor at least 1")
    if scaling in ("bands", "ramp") and original < 1:
        raise ValueError(f"scaling {scaling!r} needs the original length")
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling in ("none", "base"):
        return f, 1.0
    if scaling == "linear":
        return [v / factor for v in f], 1.0
    low, high = 1.0 if low is None else low, (4.0 if scaling == "bands" else 32.0) if high is None else high
    if not 0 < low < high:
        raise ValueError("low must be above 0 and below high")
    if scaling == "bands":
        share = [min(max((original * v / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for v in f]
        return [v * s + v / factor * (1 - s) for v, s in zip(f, share)], 1.0
    if scaling == "ramp":
        at = [rot_dim * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (high, low)]
        first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot_dim - 1)
        ramp = [min(max((i - first) / max(last - first, 0.001), 0.0), 1.0) for i in range(rot_dim // 2)]
        return [v * (1 - r) + v / factor * r for v, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    raise ValueError(f"unknown scaling {scaling!r}")


class Rotary:
    """The rotation of heads of head_dim by positions: `frequencies` (radians a position, one a pair; any sequence or tensor,
    taken in 64 bits: scaled_frequencies gives those of long contexts) for the first 2 len(frequencies) values of a head, in
    pairs (i, i + half) or, interleaved, (2i, 2i + 1); turned values are multiplied by `factor`. Laid out once."""

    def __init__(self, frequencies, head_dim: int, interleaved: bool = False, factor: float = 1.0, device=None):
        f = [float(v) for v in (frequencies.tolist() if hasattr(frequencies, "tolist") else frequencies)]
        if not f or 2 * len(f) > head_dim or not all(math.isfinite(v) for v in f):
            raise ValueError("frequencies must be finite, one to head_dim / 2 of them")
        if not (math.isfinite(factor) and factor > 0):
            raise ValueError("factor must be positive")
        # 2^64 times the turns a position, modulo 2^64, in integers: off by the last bit at most
        turns = [((n * _TURN // d >> 95) + 1 >> 1) % 2 ** 64 for n, d in (v.as_integer_ratio() for v in f)]
        device = device or torch.device("cuda", torch.cuda.current_device())
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64).to(device)
        self.head_dim, self.rot_dim, self.interleaved, self.factor = head_dim, 2 * len(f), bool(interleaved), float(factor)


def twell_rope_fwd(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, rotary: Rotary,
                   q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Queries and keys (or queries alone) turned by their tokens' positions: returns (q_out, k_out).

    q and k [tokens, heads, head_dim] with int32 positions [tokens], or [sequences, tokens, heads, head_dim] with positions
    [sequences, tokens] or [tokens]; bf16 or fp32, any strides with head_dim contiguous (slices of a fused projection,
    head-first tensors transposed). q_out may be q and k_out k: the call then works in place."""
    if q_out is None:
        q_out = _empty(q.shape, q.dtype, q.device, stream)
    if k_out is None and k is not None:
        k_out = _empty(k.shape, k.dtype, k.device, stream)
    code = (_native or _calls()).rope(q, k, positions, rotary.turns, rotary.factor, rotary.interleaved, rotary.head_dim, q_out,
                                      k_out, False, None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_rope_fwd")
    return q_out, k_out


def twell_rope_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], positions: torch.Tensor, rotary: Rotary,
                   q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Gradients of twell_rope_fwd's outputs to those of its inputs: the same call with the opposite turn."""
    if q_out is None:
        q_out = _empty(dq.shape, dq.dtype, dq.device, stream)
    if k_out is None and dk is not None:
        k_out = _empty(dk.shape, dk.dtype, dk.device, stream)
    code = (_native or _calls()).rope(dq, dk, positions, rotary.turns, rotary.factor, rotary.interleaved, rotary.head_dim, q_out,
                                      k_out, True, None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_rope_bwd")
    return q_out, k_out


@dataclasses.dataclass
class PagePool:
    """The pages of a cache that no sequence has (twell_page_pool in include/twell.h), for twell_kv_plan."""

    ring: torch.Tensor  # int32 [n_pages]
    state: torch.Tensor  # int32 [4]: first free cell, number of free pages, 0, 0
    page_size: int

    @staticmethod
    def full(n_pages: int, page_size: int, device=None):
        """All pages free."""
        if not 0 <= n_pages <= INT32_MAX:
            raise ValueError(f"the number of pages must fit 32 bits, not {n_pages}")
        device = device or torch.device("cuda", torch.cuda.current_device())
        return PagePool(torch.arange(n_pages, dtype=torch.int32, device=device),
                        torch.tensor([0, n_pages, 0, 0], dtype=torch.int32).to(device), page_size)


@dataclasses.dataclass
class StepPlan:
    """A step's tokens, one request after the other; int32, of a padding token -1, 0 and -1."""

    slots: torch.Tensor  # [n_tokens], for twell_kv_append
    positions: torch.Tensor  # [n_tokens], for twell_rope_fwd
    owner: torch.Tensor  # [n_tokens] the request's label, or its number
    starts: torch.Tensor  # [B + 1] where each request's tokens begin

    def per_token(self, page_table: torch.Tensor, seq_lens: torch.Tensor, stream=None):
        """(page_table [n_tokens, max_pages], seq_lens [n_tokens]): for each token its request's row of page_table [B, max_pages] and
        how many of its tokens there are up to this one, of the lengths [B] after the step; 0 where a token has no slot. What
        twell_paged_attn_decode and DecoderLayer.decode take, whose row i is token i, of a step in which some requests have
        no new token, or several."""
        B, n = page_table.shape[0], self.slots.numel()
        if self.starts.numel() != B + 1 or seq_lens.numel() != B:
            raise ValueError(f"the plan is of {self.starts.numel() - 1} requests, not {B} and {seq_lens.numel()}")
        with under_stream(stream):
            if B == 0:
                return page_table.new_zeros((n, page_table.shape[1])), seq_lens.new_zeros(n)
            token = torch.arange(n, dtype=torch.int32, device=self.starts.device)
            owner = (torch.searchsorted(self.starts, token, right=True) - 1).clamp_(max=B - 1)
            behind = self.starts[owner + 1] - 1 - token  # tokens of its request behind it
            return page_table[owner], torch.where(self.slots >= 0, seq_lens[owner] - behind, 0)


def twell_kv_plan(pool: PagePool, page_table: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor, n_tokens: int,
                  labels: Optional[torch.Tensor] = None, plan: Optional[StepPlan] = None,
                  seq_lens_out: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None, status=None,
                  stream=None) -> StepPlan:
    """The plan of a step, made on the device: new_lens [B] new tokens of each request (0: none, -1: it has ended) behind the
    seq_lens [B] that it has, in n_tokens rows (those past the last request's are padding).

    New tokens get pages from the pool, which are written into page_table [B, max_pages]; the pages of requests that have
    ended go back to it. seq_lens becomes the lengths after the step (0 for those that have ended) and the pool's state what
    is left, both in place unless seq_lens_out and state_out are given. labels [B], an adapter's number say, become
    the owner of their requests' tokens. All int32. A request whose tokens find no pages, row or place gets none: its tokens'
    slots are -1, its length stays, and TWELL_ERR_POOL_EMPTY or TWELL_ERR_DEVICE_CHECK is recorded in the status."""
    if plan is None:
        dev = pool.ring.device
        if not 0 <= n_tokens <= INT32_MAX:
            raise ValueError(f"n_tokens must fit 32 bits, not {n_tokens}")
        plan = StepPlan(*(_empty((n_tokens,), torch.int32, dev, stream) for _ in range(3)),
                        _empty((page_table.shape[0] + 1,), torch.int32, dev, stream))
    elif plan.slots.numel() != n_tokens:
        raise ValueError(f"the plan has {plan.slots.numel()} rows, not {n_tokens}")
    code = (_native or _calls()).kv_plan(pool.ring, pool.state, pool.page_size, page_table, seq_lens, new_lens, labels, plan.slots,
                                         plan.positions, plan.owner, plan.starts,
                                         seq_lens if seq_lens_out is None else seq_lens_out,
                                         pool.state if state_out is None else state_out,
                                         _status(status, pool.ring.get_device()), None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_kv_plan")
    return plan


@dataclasses.dataclass
class Adapters:
    """Low-rank adapters of one projection (twell_adapters in include/twell.h): adapter i adds scale[i] b[i] a[i] to its
    weights, of which the first ranks[i] rows of a[i] and columns of b[i] count (ranks None: all)."""

    a: torch.Tensor  # bf16 [n_adapters, rank, k]
    b: torch.Tensor  # bf16 [n_adapters, n, rank]
    scale: torch.Tensor  # fp32 [n_adapters]
    ranks: Optional[torch.Tensor] = None  # int32 [n_adapters]


def twell_lora_add(y: torch.Tensor, x: torch.Tensor, adapters: Adapters, ids: torch.Tensor,
                   out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, status=None,
                   stream=None) -> torch.Tensor:
    """Each token's own adapter added to a shared projection's output: y [N, n] += scale b a x [N, k] of adapter ids [N] (int32,
    any order; -1: none), in place, or into `out` when it is given. bf16, rows of any stride (slices of a fused
    projection); up to 2^20 tokens. ws as in twell_paged_attn_decode."""
    if out is None:
        out = y
    code = (_native or _calls()).lora_add(y, x, adapters.a, adapters.b, adapters.scale, adapters.ranks, ids, out, ws,
                                          _status(status, x.get_device()), None if stream is None else stream.cuda_stream)
    if code:
        _check(code, "twell_lora_add")
    return out
