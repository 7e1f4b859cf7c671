"""ctypes binding of liblily_moe.so (include/lily_moe.h), argument marshalling only.

Every function here has the name of the C entry point it calls.  Tensors are
passed as device pointers (``tensor.data_ptr()``), streams as the raw CUDA
stream handle of a ``torch.cuda.Stream`` (default: the current stream).  Every
step of the layer runs in the library's CUDA kernels; there is no Python or CPU
fallback: if the library cannot be loaded, the first call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Dict, Optional, Sequence

import torch

from . import build as _build

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None

LILY_OK = 0
STATUS_NAMES = {0: "LILY_OK", -1: "LILY_ERR_INVALID", -2: "LILY_ERR_UNSUPPORTED", -3: "LILY_ERR_MISALIGNED",
                -4: "LILY_ERR_WORKSPACE", -5: "LILY_ERR_LAUNCH", -6: "LILY_ERR_DEVICE_TIMEOUT",
                -7: "LILY_ERR_DEVICE_INDEX", -8: "LILY_ERR_SCRATCH_LIMIT", -9: "LILY_ERR_DEVICE_RANGE"}


class LilyError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        detail = f"; {lily_moe_last_error_detail()}" if code == -5 else ""
        super().__init__(f"{fn} returned {code} ({STATUS_NAMES.get(code, '?')}: {lily_moe_status_string(code)}){detail}")


class lily_moe_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "d", "E", "top_k", "I", "I_shared", "group", "block_rows")]


class lily_q4(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p)]
    # not part of the C struct: the matrix's size and CUDA device, as make_q4 found them
    rows = K = device = -1


class lily_moe_weights(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p)] + [
        (n, lily_q4) for n in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")]


class lily_moe_routing(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("logits", "topk_idx", "topk_w", "counts", "offsets", "perm", "block_map", "n_blocks")]


class lily_attn_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H_q", "H_kv", "D", "block_size", "max_blocks")]


class lily_gdn_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H_k", "H_v", "d_k", "d_v")]


class lily_kvq_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H_q", "H_kv", "D", "block_size", "max_blocks", "bits")]


class lily_kvq_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_q", "k_sb", "v_q", "v_sb")] + [
        (n, ctypes.c_int64) for n in ("n_blocks", "code_bytes")]
    # not part of the C struct: CUDA device of the arrays, and the shape of a block's codes (None: not known)
    device = 0
    block = None


class lily_norm_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "H", "d", "x_type", "h_type", "w_type")]


class lily_q4_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "rows", "K", "x_type", "out_type")]


class lily_rope_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "H_q", "H_k", "D", "rot", "interleaved")]


class lily_rope_scaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32)] + [(n, ctypes.c_double) for n in ("theta", "factor", "original", "low", "high")]


class lily_draft_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "N", "V")]


class lily_moe_decode_trace(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("logits", "topk_idx", "topk_w")]


def _configure(L: ctypes.CDLL) -> ctypes.CDLL:
    """Declares the argument and return types of every entry point."""
    P, S, I32, I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
    PS, PW, PR = ctypes.POINTER(lily_moe_shape), ctypes.POINTER(lily_moe_weights), ctypes.POINTER(lily_moe_routing)
    L.lily_moe_version.restype = I32
    L.lily_moe_status_string.restype = ctypes.c_char_p
    L.lily_moe_status_string.argtypes = [I32]
    L.lily_moe_last_error_detail.restype = ctypes.c_char_p
    L.lily_moe_last_error_detail.argtypes = []
    L.lily_moe_check_shape.argtypes = [PS]
    L.lily_moe_block_capacity.restype = I64
    L.lily_moe_block_capacity.argtypes = [PS]
    L.lily_moe_workspace_bytes.restype = S
    L.lily_moe_workspace_bytes.argtypes = [PS, ctypes.c_int32]
    L.lily_moe_route.argtypes = [PS, PW, P, PR, P, S, P]
    L.lily_moe_grouped_gemm.argtypes = [PS, PW, P, PR, P, P, S, P]
    L.lily_moe_forward.argtypes = [PS, PW, P, P, PR, P, S, P]
    L.lily_moe_forward_timed.argtypes = [PS, PW, P, P, PR, P, S, P, ctypes.POINTER(ctypes.c_void_p)]
    L.lily_moe_decode.argtypes = [PS, ctypes.c_int32, PW, P, P, P, ctypes.POINTER(lily_moe_decode_trace), P, S, P]
    L.lily_moe_route_noalloc.argtypes = [PS, PW, P, PR, P, P]
    PA = ctypes.POINTER(lily_attn_shape)
    L.lily_attn_workspace_bytes.restype = S
    L.lily_attn_workspace_bytes.argtypes = [PA]
    L.lily_attn_decode.argtypes = [PA, P, P, P, I64, P, P, ctypes.c_float, P, P, S, P]
    L.lily_attn_decode.restype = I32
    L.lily_gdn_scan.argtypes = [ctypes.POINTER(lily_gdn_shape), P, P, P, P, P, P, ctypes.c_float, P, P, P]
    L.lily_gdn_scan.restype = I32
    PQ, PC = ctypes.POINTER(lily_kvq_shape), ctypes.POINTER(lily_kvq_cache)
    L.lily_kvq_workspace_bytes.restype = S
    L.lily_kvq_workspace_bytes.argtypes = [PQ, ctypes.c_int32]
    for n in ("lily_kvq_append", "lily_kvq_read"):
        getattr(L, n).argtypes = [PQ, PC, P, I64, P, I64, ctypes.c_int32, P, P, P, P, S, P]
    L.lily_kvq_attn_decode.argtypes = [PQ, PC, P, I64, P, P, ctypes.c_float, P, P, S, P]
    L.lily_kvq_attn_prefill.argtypes = [PQ, PC, P, I64, ctypes.c_int32, P, P, P, ctypes.c_float, P, P, S, P]
    for n in ("lily_kvq_append", "lily_kvq_read", "lily_kvq_attn_decode", "lily_kvq_attn_prefill"):
        getattr(L, n).restype = I32
    F = ctypes.c_float
    L.lily_rms_norm.argtypes = [ctypes.POINTER(lily_norm_shape), P, I64, P, P, P, F, F, P, P, P, P]
    L.lily_q4_matvec.argtypes = [ctypes.POINTER(lily_q4_shape), ctypes.POINTER(lily_q4), P, I64, P, P, P]
    L.lily_rope.argtypes = [ctypes.POINTER(lily_rope_shape), P, I64, P, I64, P, P, F, P, I64, P, I64, P]
    L.lily_rope_frequencies.argtypes = [ctypes.POINTER(lily_rope_scaling), ctypes.c_int32, P]
    L.lily_rope_table.argtypes = [P, ctypes.c_int32, P]
    L.lily_draft_verify.argtypes = [ctypes.POINTER(lily_draft_shape), P, I64, P, I64, P, P, P, P, P, P, P, S, P]
    for n in ("lily_rms_norm", "lily_q4_matvec", "lily_rope", "lily_rope_frequencies", "lily_rope_table", "lily_draft_verify"):
        getattr(L, n).restype = I32
    L.lily_moe_device_status.argtypes = [P, P]
    L.lily_moe_clear_status.argtypes = [P, P]
    for n in ("lily_moe_check_shape", "lily_moe_route", "lily_moe_grouped_gemm", "lily_moe_forward",
              "lily_moe_forward_timed", "lily_moe_decode", "lily_moe_device_status", "lily_moe_route_noalloc",
              "lily_moe_clear_status"):
        getattr(L, n).restype = I32
    return L


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Loads the in-tree library (building it first if needed)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or _build.build()
            if not os.path.exists(p):
                raise OSError(f"liblily_moe.so not found at {p}")
            _lib = _configure(ctypes.CDLL(p))
    return _lib


_variants: Dict[str, ctypes.CDLL] = {}


def load_variant(variant: str) -> ctypes.CDLL:
    """Loads a test-only build variant of the library (see build.VARIANTS) as a
    separate library with its own kernels and static device data."""
    with _lock:
        if variant not in _variants:
            _variants[variant] = _configure(ctypes.CDLL(_build.build(variants=(variant,))))
    return _variants[variant]


# ------------------------------------------------------------------ marshalling helpers
def _ptr(t) -> Optional[int]:
    """Device address of a tensor argument (None stays NULL; an int is taken as a
    raw device pointer).  Tensors must be dense CUDA tensors: the library reads
    them as row-major device arrays and cannot tell a host address from a device one."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device} (shape {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"expected a contiguous tensor, got strides {t.stride()} (shape {tuple(t.shape)})")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int) -> int:
    if rc != LILY_OK:
        raise LilyError(fn, rc)
    return rc


def make_shape(T: int, d: int, E: int = 256, top_k: int = 8, I: int = 512, I_shared: Optional[int] = None,
               group: int = 64, block_rows: int = 128) -> lily_moe_shape:
    return lily_moe_shape(T, d, E, top_k, I, I if I_shared is None else I_shared, group, block_rows)


def make_weights(layer: Dict[str, torch.Tensor]) -> lily_moe_weights:
    """Weight struct of one layer from a dict of device tensors (names as in
    bit_grouped_expert_top_gb300.inputs.make_layer).  The caller keeps the
    tensors alive."""
    w = lily_moe_weights()
    w.router_w = _ptr(layer["router_w"])
    w.router_bias = _ptr(layer.get("router_bias"))
    for n in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down"):
        setattr(w, n, lily_q4(_ptr(layer[n + "_q"]), _ptr(layer[n + "_s"]), _ptr(layer[n + "_b"])))
    return w


def make_routing(tensors: Dict[str, torch.Tensor]) -> lily_moe_routing:
    r = lily_moe_routing()
    for n, _ in lily_moe_routing._fields_:
        setattr(r, n, _ptr(tensors.get(n)))
    return r


def alloc_routing(shape: lily_moe_shape, device="cuda", with_logits: bool = True) -> Dict[str, torch.Tensor]:
    """Caller-owned routing tables for `shape` (torch allocates them)."""
    T, E, k = shape.T, shape.E, shape.top_k
    cap = lily_moe_block_capacity(shape)
    out = {
        "topk_idx": torch.empty((T, k), dtype=torch.int32, device=device),
        "topk_w": torch.empty((T, k), dtype=torch.float32, device=device),
        "counts": torch.empty((E,), dtype=torch.int32, device=device),
        "offsets": torch.empty((E + 1,), dtype=torch.int32, device=device),
        "perm": torch.empty((T * k,), dtype=torch.int32, device=device),
        "block_map": torch.empty((max(cap, 1), 3), dtype=torch.int32, device=device),
        "n_blocks": torch.empty((1,), dtype=torch.int32, device=device),
    }
    if with_logits:
        out["logits"] = torch.empty((T, E), dtype=torch.float32, device=device)
    return out


def alloc_workspace(shape: lily_moe_shape, n_layers_decode: int = 0, device="cuda") -> torch.Tensor:
    n = lily_moe_workspace_bytes(shape, n_layers_decode)
    if n == 0:
        raise LilyError("lily_moe_workspace_bytes", -2)
    ws = torch.zeros((n,), dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


# ------------------------------------------------------------------ entry points (same names as the C ABI)
def lily_moe_version() -> int:
    return load().lily_moe_version()


def lily_moe_status_string(code: int) -> str:
    return load().lily_moe_status_string(int(code)).decode()


def lily_moe_last_error_detail() -> str:
    return load().lily_moe_last_error_detail().decode()


def lily_moe_check_shape(shape: lily_moe_shape) -> int:
    return load().lily_moe_check_shape(ctypes.byref(shape))


def lily_moe_block_capacity(shape: lily_moe_shape) -> int:
    return load().lily_moe_block_capacity(ctypes.byref(shape))


def lily_moe_workspace_bytes(shape: lily_moe_shape, n_layers_decode: int = 0) -> int:
    return load().lily_moe_workspace_bytes(ctypes.byref(shape), int(n_layers_decode))


def lily_moe_route(shape, weights, x, routing, ws, stream=None, *, check: bool = True) -> int:
    rc = load().lily_moe_route(ctypes.byref(shape), ctypes.byref(weights), _ptr(x), ctypes.byref(routing),
                               _ptr(ws), ws.numel() if isinstance(ws, torch.Tensor) else 0, _stream(stream))
    return _check("lily_moe_route", rc) if check else rc


def lily_moe_grouped_gemm(shape, weights, x, routing, out, ws, stream=None, *, check: bool = True) -> int:
    rc = load().lily_moe_grouped_gemm(ctypes.byref(shape), ctypes.byref(weights), _ptr(x), ctypes.byref(routing),
                                      _ptr(out), _ptr(ws), ws.numel() if isinstance(ws, torch.Tensor) else 0,
                                      _stream(stream))
    return _check("lily_moe_grouped_gemm", rc) if check else rc


def lily_moe_forward(shape, weights, x, out, ws, routing=None, stream=None, *, check: bool = True) -> int:
    rc = load().lily_moe_forward(ctypes.byref(shape), ctypes.byref(weights), _ptr(x), _ptr(out),
                                 None if routing is None else ctypes.byref(routing), _ptr(ws),
                                 ws.numel() if isinstance(ws, torch.Tensor) else 0, _stream(stream))
    return _check("lily_moe_forward", rc) if check else rc


def lily_moe_forward_timed(shape, weights, x, out, ws, events: Sequence[torch.cuda.Event], routing=None,
                           stream=None, *, check: bool = True) -> int:
    """As lily_moe_forward, recording 6 events (start, after router GEMM, after
    routing tables, after the routing-order copy of x, after gate/up, after down)."""
    assert len(events) == 6
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event on first record
            e.record(torch.cuda.current_stream() if stream is None else stream)
    arr = (ctypes.c_void_p * 6)(*[e.cuda_event for e in events])
    rc = load().lily_moe_forward_timed(ctypes.byref(shape), ctypes.byref(weights), _ptr(x), _ptr(out),
                                       None if routing is None else ctypes.byref(routing), _ptr(ws),
                                       ws.numel() if isinstance(ws, torch.Tensor) else 0, _stream(stream), arr)
    return _check("lily_moe_forward_timed", rc) if check else rc


def lily_moe_decode(shape, layers: Sequence[lily_moe_weights], x, out, ws, x_next=None,
                    trace: Optional[Dict[str, torch.Tensor]] = None, stream=None, *, check: bool = True) -> int:
    arr = (lily_moe_weights * len(layers))(*layers)
    tr = None
    if trace is not None:
        tr = lily_moe_decode_trace(_ptr(trace.get("logits")), _ptr(trace.get("topk_idx")), _ptr(trace.get("topk_w")))
    rc = load().lily_moe_decode(ctypes.byref(shape), len(layers), arr, _ptr(x), _ptr(out), _ptr(x_next),
                                None if tr is None else ctypes.byref(tr), _ptr(ws),
                                ws.numel() if isinstance(ws, torch.Tensor) else 0, _stream(stream))
    return _check("lily_moe_decode", rc) if check else rc


def lily_moe_device_status(ws, stream=None) -> int:
    return load().lily_moe_device_status(_ptr(ws), _stream(stream))


def lily_moe_clear_status(ws, stream=None) -> int:
    return _check("lily_moe_clear_status", load().lily_moe_clear_status(_ptr(ws), _stream(stream)))


def lily_moe_route_noalloc(shape, weights, x, routing, device_status=None, stream=None, *, check: bool = True) -> int:
    """Routing without a caller workspace: for callers that may not allocate
    device memory when they run the layer (e.g. inside another engine's fixed
    memory budget).  Scratch lives in a fixed device array owned by the
    library (T <= 8192); calls that may overlap on the GPU race.  `routing`
    must include logits; `device_status` (device int32 tensor) receives the
    call's device status."""
    rc = load().lily_moe_route_noalloc(ctypes.byref(shape), ctypes.byref(weights), _ptr(x), ctypes.byref(routing),
                                       _ptr(device_status), _stream(stream))
    return _check("lily_moe_route_noalloc", rc) if check else rc


# ------------------------------------------------------------------ decode attention
def make_attn_shape(B: int, H_q: int, H_kv: int, D: int, block_size: int, max_blocks: int) -> lily_attn_shape:
    return lily_attn_shape(B, H_q, H_kv, D, block_size, max_blocks)


def lily_attn_workspace_bytes(shape: lily_attn_shape) -> int:
    return load().lily_attn_workspace_bytes(ctypes.byref(shape))


def alloc_attn_workspace(shape: lily_attn_shape, device="cuda") -> torch.Tensor:
    n = lily_attn_workspace_bytes(shape)
    if n == 0:
        raise ValueError("unsupported attention shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def lily_attn_decode(shape: lily_attn_shape, q, k_cache, v_cache, block_table, seq_lens, out, ws,
                     scale: Optional[float] = None, stream=None, *, check: bool = True) -> int:
    """Grouped-query decode attention over a fixed-block KV cache (see
    include/lily_moe.h).  scale defaults to 1/sqrt(D)."""
    if scale is None:
        scale = 1.0 / math.sqrt(shape.D)
    n_blocks = k_cache.shape[0] if isinstance(k_cache, torch.Tensor) else 0
    rc = load().lily_attn_decode(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), n_blocks,
                                 _ptr(block_table), _ptr(seq_lens), float(scale), _ptr(out), _ptr(ws),
                                 ws.numel() if isinstance(ws, torch.Tensor) else 0, _stream(stream))
    return _check("lily_attn_decode", rc) if check else rc


# ------------------------------------------------------------------ quantised KV cache
def make_kvq_shape(B: int, H_q: int, H_kv: int, D: int, block_size: int, max_blocks: int, bits: int = 4) -> lily_kvq_shape:
    return lily_kvq_shape(B, H_q, H_kv, D, block_size, max_blocks, bits)


def alloc_kvq_cache(shape: lily_kvq_shape, n_blocks: int, device="cuda") -> Dict[str, torch.Tensor]:
    """The four arrays of a cache of n_blocks blocks (codes uint8 and parameters
    bf16 of K and V, zeroed); hand them to make_kvq_cache."""
    if lily_kvq_workspace_bytes(shape) == 0:
        raise ValueError("unsupported quantised-cache shape")
    lead = (n_blocks, shape.H_kv, shape.D // 64, shape.block_size)
    out = {}
    for n in ("k", "v"):
        out[n + "_q"] = torch.zeros(lead + (8 * shape.bits,), dtype=torch.uint8, device=device)
        out[n + "_sb"] = torch.zeros(lead + (2,), dtype=torch.bfloat16, device=device)
    return out


def make_kvq_cache(tensors: Dict[str, torch.Tensor]) -> lily_kvq_cache:
    """Cache struct of the four arrays of alloc_kvq_cache (codes [n_blocks][H_kv]
    [D/64][block_size][8 bits], parameters [...][2]).  The caller keeps the
    tensors alive."""
    k_q = tensors["k_q"]
    for n in ("k", "v"):
        q, sb = tensors[n + "_q"], tensors[n + "_sb"]
        if q.dtype != torch.uint8 or sb.dtype != torch.bfloat16:
            raise ValueError(f"{n}_q must be uint8 and {n}_sb bfloat16, got {q.dtype} and {sb.dtype}")
        if q.dim() != 5 or q.shape != k_q.shape or sb.shape != q.shape[:-1] + (2,):
            raise ValueError(f"cache arrays of unlike shapes: {n}_q {tuple(q.shape)}, {n}_sb {tuple(sb.shape)}")
        if q.device != k_q.device or sb.device != k_q.device:
            raise ValueError("cache arrays on different devices")
    cache = lily_kvq_cache(_ptr(k_q), _ptr(tensors["k_sb"]), _ptr(tensors["v_q"]), _ptr(tensors["v_sb"]),
                           k_q.shape[0], k_q.numel())
    cache.device = k_q.get_device()
    cache.block = tuple(k_q.shape[1:])
    return cache


def lily_kvq_workspace_bytes(shape: lily_kvq_shape, n_query: int = 0) -> int:
    return load().lily_kvq_workspace_bytes(ctypes.byref(shape), int(n_query))


def alloc_kvq_workspace(shape: lily_kvq_shape, n_query: int = 0, device="cuda") -> torch.Tensor:
    """Workspace of the lily_kvq_* calls; n_query: the most query tokens of a
    lily_kvq_attn_prefill call (0: none)."""
    n = lily_kvq_workspace_bytes(shape, n_query)
    if n == 0:
        raise ValueError("unsupported quantised-cache shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


# A call's tensors are checked in one flat condition, as a decode step of short sequences takes
# the GPU less time than a careless wrapper takes the host; where it does not hold,
# the functions below find out why and raise.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the current stream without a Stream object
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # for callers that hold a CUDA tensor
_BF16, _I32, _U8 = torch.bfloat16, torch.int32, torch.uint8


def _need(ok: bool, message: str) -> None:
    if not ok:
        raise ValueError(message)


def _need_device(name: str, t, cache) -> int:
    """The library launches on the current device: a tensor (or a cache) elsewhere is refused."""
    dev = t.get_device()
    _need(dev >= 0, f"expected a CUDA tensor, got one on {t.device} ({name}, shape {tuple(t.shape)})")
    _need(dev == torch.cuda.current_device(),
          f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    _need(cache.device == dev, f"the cache is on cuda:{cache.device}, {name} on cuda:{dev}")
    return dev


def _need_dense(name: str, t, dtype, n: int, dev: int) -> None:
    _need(t.is_cuda, f"expected a CUDA tensor, got one on {t.device} ({name}, shape {tuple(t.shape)})")
    _need(t.dtype is dtype and t.numel() >= n and t.get_device() == dev and t.is_contiguous(),
          f"{name}: expected {n} contiguous {dtype} on cuda:{dev}, got {t.dtype} {list(t.shape)} with "
          f"strides {t.stride()} on {t.device}")


def _need_tokens(name: str, t, heads: int, D: int, dev: int) -> None:
    _need(t.dtype is _BF16 and t.dim() == 3 and t.shape[1] == heads and t.shape[2] == D,
          f"{name}: expected bfloat16 [n][{heads}][{D}], got {t.dtype} {list(t.shape)}")
    _need(t.get_device() == dev, f"{name}: expected a CUDA tensor on cuda:{dev}, got one on {t.device}")
    _need(t.stride(2) == 1 and (t.stride(1) == D or heads == 1),
          f"{name}: the heads of a token must be contiguous, got strides {t.stride()}")


def _need_block(shape, cache) -> None:
    """A cache of other heads, blocks or bits can have as many bytes of codes, but other ones of parameters."""
    block = (shape.H_kv, shape.D >> 6, shape.block_size, 8 * shape.bits)
    _need(cache.block in (None, block),
          f"cache: blocks of {cache.block} (KV heads, groups, tokens, bytes of codes), the shape has {block}")


def _need_table(t, shape, dev: int) -> None:
    _need(t.shape == (shape.B, shape.max_blocks),
          f"block_table: expected [{shape.B}][{shape.max_blocks}], got {list(t.shape)}")
    _need_dense("block_table", t, _I32, shape.B * shape.max_blocks, dev)


def _launch_stream(stream, dev: int):
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def _kvq_copy(fn: str, shape, cache, k, v, cu, starts, block_table, ws, stream, check: bool) -> int:
    B, H, D = shape.B, shape.H_kv, shape.D
    dev, size, sk, sv = k.get_device(), k.shape, k.stride(), v.stride()
    if not (k.dtype is _BF16 and v.dtype is _BF16 and v.shape == size and len(size) == 3 and size[1] == H and size[2] == D
            and sk[2] == 1 and sv[2] == 1 and (H == 1 or (sk[1] == D and sv[1] == D))
            and cu.dtype is _I32 and cu.numel() > B and cu.is_contiguous()
            and starts.dtype is _I32 and starts.numel() >= B and starts.is_contiguous()
            and block_table.dtype is _I32 and block_table.shape == (B, shape.max_blocks) and block_table.is_contiguous()
            and ws.dtype is _U8 and ws.is_contiguous()
            and cache.block in (None, (H, D >> 6, shape.block_size, 8 * shape.bits))
            and dev >= 0 and dev == _current_device() == cache.device == v.get_device() == cu.get_device()
            == starts.get_device() == block_table.get_device() == ws.get_device()):
        _need_block(shape, cache)
        _need(k.dtype is _BF16, f"k: expected bfloat16, got {k.dtype}")
        _need(v.shape[0] == k.shape[0], f"k has {k.shape[0]} tokens, v {v.shape[0]}")
        dev = _need_device("k", k, cache)
        _need_tokens("k", k, H, D, dev)
        _need_tokens("v", v, H, D, dev)
        _need_dense("cu", cu, _I32, B + 1, dev)
        _need_dense("starts", starts, _I32, B, dev)
        _need_table(block_table, shape, dev)
        _need_dense("ws", ws, _U8, 1, dev)
        raise ValueError("tensors on different devices")
    N = size[0]
    rc = getattr(_lib or load(), fn)(
        ctypes.byref(shape), ctypes.byref(cache), k.data_ptr(), sk[0] if N > 1 else H * D, v.data_ptr(),
        sv[0] if N > 1 else H * D, N, cu.data_ptr(), starts.data_ptr(), block_table.data_ptr(), ws.data_ptr(), ws.numel(),
        _launch_stream(stream, dev))
    return _check(fn, rc) if check else rc


def lily_kvq_append(shape: lily_kvq_shape, cache: lily_kvq_cache, k, v, cu_new, starts, block_table, ws, stream=None,
                    *, check: bool = True) -> int:
    """Quantises k and v (bf16 [N][H_kv][D], any token stride) into the cache
    (see include/lily_moe.h)."""
    return _kvq_copy("lily_kvq_append", shape, cache, k, v, cu_new, starts, block_table, ws, stream, check)


def lily_kvq_read(shape: lily_kvq_shape, cache: lily_kvq_cache, k, v, cu, starts, block_table, ws, stream=None,
                  *, check: bool = True) -> int:
    """Reads cached tokens back into k and v (bf16 [N][H_kv][D], any token stride)."""
    return _kvq_copy("lily_kvq_read", shape, cache, k, v, cu, starts, block_table, ws, stream, check)


def _kvq_attention(shape, cache, q, cu_q, block_table, seq_lens, out, ws, scale, stream):
    """The checks of both attentions (cu_q None: decode).  Device, stream, token stride of q and the scale."""
    B, H, D = shape.B, shape.H_q, shape.D
    dev, size, sq = q.get_device(), q.shape, q.stride()
    if not (q.dtype is _BF16 and len(size) == 3 and size[1] == H and size[2] == D and sq[2] == 1 and (H == 1 or sq[1] == D)
            and block_table.dtype is _I32 and block_table.shape == (B, shape.max_blocks) and block_table.is_contiguous()
            and seq_lens.dtype is _I32 and seq_lens.numel() >= B and seq_lens.is_contiguous()
            and out.dtype is _BF16 and out.numel() >= size[0] * H * D and out.is_contiguous()
            and ws.dtype is _U8 and ws.is_contiguous()
            and cache.block in (None, (shape.H_kv, D >> 6, shape.block_size, 8 * shape.bits))
            and dev >= 0 and dev == _current_device() == cache.device == block_table.get_device() == seq_lens.get_device()
            == out.get_device() == ws.get_device()
            and (size[0] == B if cu_q is None else cu_q.dtype is _I32 and cu_q.numel() > B and cu_q.is_contiguous()
                 and cu_q.get_device() == dev)):
        _need_block(shape, cache)
        _need(q.dtype is _BF16 and q.dim() == 3 and q.shape[1] == H and q.shape[2] == D,
              f"q: expected bfloat16 [n][{H}][{D}], got {q.dtype} {list(q.shape)}")
        dev = _need_device("q", q, cache)
        _need_tokens("q", q, H, D, dev)
        if cu_q is None:
            _need(q.shape[0] == B, f"q: expected {B} sequences, got {q.shape[0]}")
        else:
            _need_dense("cu_q", cu_q, _I32, B + 1, dev)
        _need_table(block_table, shape, dev)
        _need_dense("seq_lens", seq_lens, _I32, B, dev)
        _need_dense("out", out, _BF16, q.shape[0] * H * D, dev)
        _need_dense("ws", ws, _U8, 1, dev)
        raise ValueError("tensors on different devices")
    return _launch_stream(stream, dev), sq[0] if size[0] > 1 else H * D, D ** -0.5 if scale is None else scale


def lily_kvq_attn_decode(shape: lily_kvq_shape, cache: lily_kvq_cache, q, block_table, seq_lens, out, ws,
                         scale: Optional[float] = None, stream=None, *, check: bool = True) -> int:
    """Decode attention over the quantised cache (see include/lily_moe.h): q and
    out bf16 [B][H_q][D].  scale defaults to 1/sqrt(D)."""
    stream, stride, scale = _kvq_attention(shape, cache, q, None, block_table, seq_lens, out, ws, scale, stream)
    rc = (_lib or load()).lily_kvq_attn_decode(
        ctypes.byref(shape), ctypes.byref(cache), q.data_ptr(), stride, block_table.data_ptr(), seq_lens.data_ptr(), scale,
        out.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    return _check("lily_kvq_attn_decode", rc) if check else rc


def lily_kvq_attn_prefill(shape: lily_kvq_shape, cache: lily_kvq_cache, q, cu_q, block_table, seq_lens, out, ws,
                          scale: Optional[float] = None, stream=None, *, check: bool = True) -> int:
    """Causal attention of a chunk of query tokens per sequence (q, out bf16
    [N][H_q][D], rows by cu_q) over the quantised cache that already holds the
    chunk's keys.  scale defaults to 1/sqrt(D)."""
    _need(cu_q is not None, "cu_q: expected a tensor")
    stream, stride, scale = _kvq_attention(shape, cache, q, cu_q, block_table, seq_lens, out, ws, scale, stream)
    rc = (_lib or load()).lily_kvq_attn_prefill(
        ctypes.byref(shape), ctypes.byref(cache), q.data_ptr(), stride, q.shape[0], cu_q.data_ptr(), block_table.data_ptr(),
        seq_lens.data_ptr(), scale, out.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    return _check("lily_kvq_attn_prefill", rc) if check else rc


# ------------------------------------------------------------------ Gated DeltaNet scan
def lily_gdn_scan(q, k, v, alpha, beta, out, state_out, state_in=None, scale: Optional[float] = None,
                  stream=None, *, check: bool = True) -> int:
    """Gated DeltaNet scan over the T tokens of q/k [T][H_k][d_k], v [T][H_v][d_v]
    (see include/lily_moe.h).  scale defaults to 1/sqrt(d_k)."""
    T, H_k, d_k = q.shape
    _, H_v, d_v = v.shape
    shape = lily_gdn_shape(T, H_k, H_v, d_k, d_v)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    rc = load().lily_gdn_scan(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state_in),
                              float(scale), _ptr(out), _ptr(state_out), _stream(stream))
    return _check("lily_gdn_scan", rc) if check else rc


# ------------------------------------------------------------------ around the attention and the expert layers
_F32, _E4M3, _I64 = torch.float32, torch.float8_e4m3fn, torch.int64


def _need_here(name: str, t) -> int:
    """Device of a call's first tensor, which has to be the current one."""
    dev = t.get_device()
    _need(dev >= 0, f"expected a CUDA tensor, got one on {t.device} ({name}, shape {tuple(t.shape)})")
    _need(dev == torch.cuda.current_device(),
          f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _need_type(name: str, t, *types) -> None:
    _need(t.dtype in types, f"{name}: expected {' or '.join(str(x) for x in types)}, got {t.dtype}")


def _need_array(name: str, t, dtype, shape, dev: int) -> None:
    """A dense tensor of just this shape and type on the call's device."""
    _need(t.is_cuda, f"expected a CUDA tensor, got one on {t.device} ({name}, shape {tuple(t.shape)})")
    _need(t.dtype is dtype and tuple(t.shape) == tuple(shape) and t.get_device() == dev and t.is_contiguous(),
          f"{name}: expected contiguous {dtype} {list(shape)} on cuda:{dev}, got {t.dtype} {list(t.shape)} with "
          f"strides {t.stride()} on {t.device}")


def _need_int32(*sizes) -> None:
    """ctypes would pass the low 32 bits of larger ones."""
    _need(max(sizes) < 1 << 31, f"sizes of more than 32 bits: {list(sizes)}")


def lily_rms_norm(x, weight=None, y=None, y8=None, y8_scale=None, residual=None, h=None, eps: float = 1e-6,
                  weight_offset: float = 0.0, stream=None, *, check: bool = True) -> int:
    """Root-mean-square norm with the residual's addition (see include/lily_moe.h): x [N][d], or [N][H][d] for the heads
    of N tokens (any token stride), bf16 or fp32; y bf16 and y8 (float8_e4m3fn, with y8_scale fp32 [..., d/64]) of x's
    shape.  The channel's factor is weight + weight_offset (weight None: weight_offset)."""
    size, dev, st, xt = x.shape, x.get_device(), x.stride(), x.dtype
    n = len(size)
    H, d = (1, size[1]) if n == 2 else (size[1], size[2]) if n == 3 else (0, 0)
    first, wt, rt = y if y is not None else y8, weight, residual  # the latter two: then their types
    if not (H > 0 and (xt is _BF16 or xt is _F32) and st[-1] == 1 and (n == 2 or H == 1 or st[1] == d) and first is not None
            and (weight is None or ((wt := weight.dtype) is _BF16 or wt is _F32) and weight.numel() == d and weight.dim() == 1
                 and weight.is_contiguous() and weight.get_device() == dev)
            and (y is None or (y.dtype is _BF16 and y.shape == size and y.is_contiguous() and y.get_device() == dev))
            and (y8 is None) == (y8_scale is None)
            and (y8 is None or (y8.dtype is _E4M3 and y8.shape == size and y8.is_contiguous() and y8.get_device() == dev
                                and d & 63 == 0 and y8_scale.dtype is _F32 and y8_scale.dim() == n and y8_scale.shape[-1] == d >> 6
                                and y8_scale.numel() == size[0] * H * (d >> 6) and y8_scale.is_contiguous()
                                and y8_scale.get_device() == dev))
            and (residual is None) == (h is None)
            and (residual is None or ((rt := residual.dtype) is _BF16 or rt is _F32) and h.dtype is rt and residual.shape == size
                 and h.shape == size and residual.is_contiguous() and h.is_contiguous() and residual.get_device() == dev
                 and h.get_device() == dev)
            and dev >= 0 and dev == _current_device()):
        _need(H > 0, f"x: expected [N][d] or [N][H][d] with H > 0, got {list(size)}")
        _need_type("x", x, _BF16, _F32)
        dev = _need_here("x", x)
        _need(st[-1] == 1 and (n == 2 or H == 1 or st[1] == d), f"x: the channels of a token must be contiguous, got strides {st}")
        _need(first is not None, "expected y or y8 (with y8_scale)")
        if weight is not None:
            _need_type("weight", weight, _BF16, _F32)
            _need_array("weight", weight, weight.dtype, (d,), dev)
        if y is not None:
            _need_array("y", y, _BF16, size, dev)
        _need((y8 is None) == (y8_scale is None), "y8 and y8_scale go together")
        if y8 is not None:
            _need(d % 64 == 0, f"y8: groups of 64 channels, x has {d}")
            _need_array("y8", y8, _E4M3, size, dev)
            _need_array("y8_scale", y8_scale, _F32, size[:-1] + (d // 64,), dev)
        _need((residual is None) == (h is None), "residual and h go together")
        if residual is not None:
            _need_type("residual", residual, _BF16, _F32)
            _need_array("residual", residual, residual.dtype, size, dev)
            _need_array("h", h, residual.dtype, size, dev)
        raise ValueError("tensors on different devices")
    N = size[0]
    if (N | H | d) >> 31:
        _need_int32(N, H, d)
    rc = (_lib or load()).lily_rms_norm(
        lily_norm_shape(N, H, d, xt is _F32, rt is _F32, wt is _F32), x.data_ptr(), st[0] if N > 1 else H * d, None if residual is None else residual.data_ptr(),
        None if h is None else h.data_ptr(), None if weight is None else weight.data_ptr(), weight_offset, eps,
        None if y is None else y.data_ptr(), None if y8 is None else y8.data_ptr(),
        None if y8_scale is None else y8_scale.data_ptr(), _launch_stream(stream, dev))
    return _check("lily_rms_norm", rc) if check else rc


def make_q4(q, scale, bias) -> lily_q4:
    """One 4-bit matrix of its codes (uint8 [rows][K/2]) and its bf16 scales and biases ([rows][K/64]); the
    caller keeps the tensors alive."""
    rows, half = q.shape if q.dim() == 2 else (0, 0)
    _need(q.dtype is _U8 and rows > 0 and half % 32 == 0 and half > 0,
          f"q: expected uint8 [rows][K/2], K a multiple of 64, got {q.dtype} {list(q.shape)}")
    dev = q.get_device()
    _need(dev >= 0 and q.is_contiguous(), f"q: expected a contiguous CUDA tensor, got strides {q.stride()} on {q.device}")
    _need_array("scale", scale, _BF16, (rows, half // 32), dev)
    _need_array("bias", bias, _BF16, (rows, half // 32), dev)
    _need_int32(rows, 2 * half)
    w = lily_q4(q.data_ptr(), scale.data_ptr(), bias.data_ptr())
    w.rows, w.K, w.device = rows, 2 * half, dev
    return w


def lily_q4_matvec(w: lily_q4, x, out, x_scale=None, stream=None, *, check: bool = True) -> int:
    """Up to 32 tokens times the 4-bit matrix of make_q4 (see include/lily_moe.h): x bf16 [T][K], or float8_e4m3fn
    with x_scale fp32 [T][K/64] (lily_rms_norm's y8); out bf16 or fp32 [T][rows]."""
    rows, K = w.rows, w.K
    dev, size, st, xt, ot = x.get_device(), x.shape, x.stride(), x.dtype, out.dtype
    if not (len(size) == 2 and size[1] == K and st[1] == 1 and (ot is _BF16 or ot is _F32) and out.shape == (size[0], rows)
            and out.is_contiguous()
            and (xt is _BF16 and x_scale is None or xt is _E4M3 and x_scale is not None and x_scale.dtype is _F32
                 and x_scale.shape == (size[0], K >> 6) and x_scale.is_contiguous() and x_scale.get_device() == dev)
            and dev >= 0 and dev == _current_device() == w.device == out.get_device()):
        _need(x.dim() == 2 and size[1] == K, f"x: expected [T][{K}], got {list(size)}")
        _need_type("x", x, _BF16, _E4M3)
        dev = _need_here("x", x)
        _need(w.device == dev, f"the matrix is on cuda:{w.device}, x on cuda:{dev}")
        _need(st[1] == 1, f"x: the channels of a token must be contiguous, got strides {st}")
        _need((xt is _E4M3) == (x_scale is not None), "x_scale goes with x in float8_e4m3fn, and only with it")
        if x_scale is not None:
            _need_array("x_scale", x_scale, _F32, (size[0], K // 64), dev)
        _need_type("out", out, _BF16, _F32)
        _need_array("out", out, ot, (size[0], rows), dev)
        raise ValueError("tensors on different devices")
    T = size[0]
    if T >> 31:
        _need_int32(T)
    rc = (_lib or load()).lily_q4_matvec(
        lily_q4_shape(T, rows, K, 2 if xt is _E4M3 else 0, ot is _F32), w, x.data_ptr(), st[0] if T > 1 else K,
        None if x_scale is None else x_scale.data_ptr(), out.data_ptr(), _launch_stream(stream, dev))
    return _check("lily_q4_matvec", rc) if check else rc


ROPE_SCALING = {"none": 0, "linear": 1, "base": 2, "parts": 3}


def rope_frequencies(rot: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0, original: float = 0.0,
                     low: float = 1.0, high: float = 32.0) -> torch.Tensor:
    """Angle of each of the rot / 2 pairs a position (fp64, on the host), scaled for contexts longer than the trained
    one: "none", "linear", "base" or "parts" (see lily_rope_frequencies in include/lily_moe.h)."""
    _need(scaling in ROPE_SCALING, f"scaling: expected one of {sorted(ROPE_SCALING)}, got {scaling!r}")
    _need_int32(rot)
    out = torch.empty(max(rot // 2, 1), dtype=torch.float64)
    c = lily_rope_scaling(ROPE_SCALING[scaling], theta, factor, original, low, high)
    _check("lily_rope_frequencies", load().lily_rope_frequencies(c, rot, out.data_ptr()))
    return out


def make_rope_table(frequencies, device="cuda") -> torch.Tensor:
    """Device table of lily_rope for these angles a position (fp64, in [0, 2 pi))."""
    f = torch.as_tensor(frequencies, dtype=torch.float64, device="cpu").contiguous()
    _need(f.dim() == 1 and f.numel() > 0, f"frequencies: expected a vector, got {list(f.shape)}")
    out = torch.empty(f.numel(), dtype=_I64)
    _check("lily_rope_table", load().lily_rope_table(f.data_ptr(), f.numel(), out.data_ptr()))
    return out.to(device)


def _rope_heads(name: str, t, dev: int) -> None:
    _need(t.dtype is _BF16 and t.dim() == 3, f"{name}: expected bfloat16 [N][H][D], got {t.dtype} {list(t.shape)}")
    _need(t.get_device() == dev, f"{name}: expected a CUDA tensor on cuda:{dev}, got one on {t.device}")
    _need(t.stride(2) == 1 and (t.stride(1) == t.shape[2] or t.shape[1] == 1),
          f"{name}: the heads of a token must be contiguous, got strides {t.stride()}")


def lily_rope(q, k, positions, table, q_out=None, k_out=None, interleaved: bool = False, amplitude: float = 1.0, stream=None,
              *, check: bool = True) -> int:
    """Rotary positions (see include/lily_moe.h): q [N][H_q][D] and k [N][H_k][D] (None: queries only) bf16 with any token
    stride; the first 2 * len(table) channels of each head turn.  q_out and k_out default to q and k (in place)."""
    if q_out is None:
        q_out = q
    if k_out is None:
        k_out = k
    dev, qs, st, so = q.get_device(), q.shape, q.stride(), q_out.stride()
    D = qs[-1]
    if k is not None and k_out is not None:
        ks, kst, kso = k.shape, k.stride(), k_out.stride()
        k_ok = (k.dtype is _BF16 and k_out.dtype is _BF16 and len(ks) == 3 and k_out.shape == ks and ks[0] == qs[0] and ks[2] == D
                and ks[1] > 0 and kst[2] == 1 and kso[2] == 1 and (ks[1] == 1 or (kst[1] == D and kso[1] == D))
                and k.get_device() == dev and k_out.get_device() == dev)
    else:
        k_ok = k is None and k_out is None
    if not (k_ok and q.dtype is _BF16 and q_out.dtype is _BF16 and len(qs) == 3 and q_out.shape == qs and st[2] == 1 and so[2] == 1
            and (qs[1] == 1 or (st[1] == D and so[1] == D)) and q_out.get_device() == dev
            and positions.dtype is _I32 and positions.shape == (qs[0],) and positions.is_contiguous() and positions.get_device() == dev
            and table.dtype is _I64 and table.dim() == 1 and table.is_contiguous() and table.get_device() == dev
            and dev >= 0 and dev == _current_device()):
        _need(q.dtype is _BF16 and q.dim() == 3, f"q: expected bfloat16 [N][H][D], got {q.dtype} {list(q.shape)}")
        dev = _need_here("q", q)
        _need((k is None) == (k_out is None), "k and k_out go together")
        for name, t, like in (("q", q, q), ("q_out", q_out, q), ("k", k, k), ("k_out", k_out, k)):
            if t is not None:
                _rope_heads(name, t, dev)
                _need(t.shape == like.shape and t.shape[0] == qs[0] and t.shape[2] == D and t.shape[1] > 0,
                      f"{name}: {list(t.shape)} beside q {list(qs)}")
        _need_array("positions", positions, _I32, (qs[0],), dev)
        _need(table.dim() == 1, f"table: expected a vector, got {list(table.shape)}")
        _need_array("table", table, _I64, table.shape, dev)
        raise ValueError("tensors on different devices")
    N, H_q = qs[0], qs[1]
    H_k = 0 if k is None else ks[1]
    rot = 2 * table.shape[0]
    if (N | H_q | H_k | D | rot) >> 31:
        _need_int32(N, H_q, H_k, D, rot)
    dense_q, dense_k = H_q * D, H_k * D
    rc = (_lib or load()).lily_rope(
        lily_rope_shape(N, H_q, H_k, D, rot, 1 if interleaved else 0), q.data_ptr(), st[0] if N > 1 else dense_q,
        None if k is None else k.data_ptr(), 0 if k is None else kst[0] if N > 1 else dense_k, positions.data_ptr(),
        table.data_ptr(), amplitude, q_out.data_ptr(), so[0] if N > 1 else dense_q, None if k is None else k_out.data_ptr(),
        0 if k is None else kso[0] if N > 1 else dense_k, _launch_stream(stream, dev))
    return _check("lily_rope", rc) if check else rc


LILY_DRAFT_WORKSPACE_BYTES = 256


def alloc_draft_workspace(device="cuda") -> torch.Tensor:
    """Workspace of lily_draft_verify (its status word)."""
    return torch.zeros(LILY_DRAFT_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def lily_draft_verify(p, q, drafts, cu, u, r, accepted, tokens, ws, stream=None, *, check: bool = True) -> int:
    """Accepts or refuses the N drafted tokens of B sequences and draws the token after them (see include/lily_moe.h): p
    fp32 [N + B][V] (the target's probabilities), q fp32 [N][V] or None (drafts without probabilities), any row
    stride; drafts int32 [N], rows by cu int32 [B+1]; uniform numbers u [N] and r [B]; accepted int32 [B] and tokens int32 [N + B]."""
    dev, ps, st = p.get_device(), p.shape, p.stride()
    B, N = r.numel(), drafts.numel()
    if not (p.dtype is _F32 and len(ps) == 2 and ps[0] == N + B and st[1] == 1 and ps[1] > 0
            and (q is None or (q.dtype is _F32 and q.shape == (N, ps[1]) and q.stride(1) == 1 and q.get_device() == dev))
            and drafts.dtype is _I32 and drafts.is_contiguous() and cu.dtype is _I32 and cu.numel() == B + 1 and cu.is_contiguous()
            and u.dtype is _F32 and u.numel() == N and u.is_contiguous() and r.dtype is _F32 and r.is_contiguous()
            and accepted.dtype is _I32 and accepted.numel() == B and accepted.is_contiguous()
            and tokens.dtype is _I32 and tokens.numel() == N + B and tokens.is_contiguous()
            and ws.dtype is _U8 and ws.is_contiguous()
            and dev >= 0 and dev == _current_device() == drafts.get_device() == cu.get_device() == u.get_device() == r.get_device()
            == accepted.get_device() == tokens.get_device() == ws.get_device()):
        _need(p.dtype is _F32 and p.dim() == 2 and ps[0] == N + B and ps[1] > 0,
              f"p: expected float32 [{N + B}][V], got {p.dtype} {list(ps)}")
        dev = _need_here("p", p)
        _need(st[1] == 1, f"p: the values of a row must be contiguous, got strides {st}")
        if q is not None:
            _need(q.dtype is _F32 and q.shape == (N, ps[1]) and q.stride(1) == 1 and q.get_device() == dev,
                  f"q: expected float32 [{N}][{ps[1]}] with contiguous rows on cuda:{dev}, got {q.dtype} {list(q.shape)} with "
                  f"strides {q.stride()} on {q.device}")
        _need_array("drafts", drafts, _I32, (N,), dev)
        _need_array("cu", cu, _I32, (B + 1,), dev)
        _need_array("u", u, _F32, (N,), dev)
        _need_array("r", r, _F32, (B,), dev)
        _need_array("accepted", accepted, _I32, (B,), dev)
        _need_array("tokens", tokens, _I32, (N + B,), dev)
        _need_dense("ws", ws, _U8, 1, dev)
        raise ValueError("tensors on different devices")
    V = ps[1]
    if (B | N | V) >> 31:
        _need_int32(B, N, V)
    rc = (_lib or load()).lily_draft_verify(
        lily_draft_shape(B, N, V), p.data_ptr(), st[0] if N + B > 1 else V, None if q is None or N == 0 else q.data_ptr(),
        V if q is None or N <= 1 else q.stride(0), drafts.data_ptr() if N else None, cu.data_ptr(), u.data_ptr() if N else None,
        r.data_ptr(), accepted.data_ptr(), tokens.data_ptr(), ws.data_ptr(), ws.numel(), _launch_stream(stream, dev))
    return _check("lily_draft_verify", rc) if check else rc
