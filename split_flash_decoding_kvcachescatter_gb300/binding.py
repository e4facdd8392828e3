"""Thin Python binding of libkvsdecode.so: argument marshalling only.

Every function here has the name of the C entry point it calls
(include/kvsdecode.h).  It checks tensor dtype/device/contiguity, reads the
sizes off the tensor shapes, passes raw device pointers and the current
CUDA stream, and raises KvsError on a non-zero status.  All compute runs
in the CUDA kernels of the library; there is no fallback of any kind: if
the library is missing or fails to load, the functions raise.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvsdecode.so")

KVS_OK = 0
KVS_ERR_NULL = 1
KVS_ERR_DIMS = 2
KVS_ERR_UNSUPPORTED = 3
KVS_ERR_ALIGN = 4
KVS_ERR_WORKSPACE = 5
KVS_ERR_LAUNCH = 6
KVS_ERR_POSITION = 7
KVS_ERR_TIMEOUT = 8
KVS_ERR_SLOT = 9
KVS_ERR_MEMORY = 10
KVS_ERR_PAGE = 11
KVS_ERR_ROWS = 12
KVS_ERR_OVERLAP = 13

# kvs_dtype values
KVS_F32, KVS_F16, KVS_BF16 = 0, 1, 2
_DTYPES = {torch.float32: KVS_F32, torch.float16: KVS_F16, torch.bfloat16: KVS_BF16}

# kvs_rope_kind values (kvs_rope_frequencies)
KVS_ROPE_PLAIN, KVS_ROPE_LINEAR, KVS_ROPE_NTK, KVS_ROPE_YARN, KVS_ROPE_BANDS = range(5)

# Every symbol include/kvsdecode.h declares.
EXPORTS = ("kvs_kv_scatter", "kvs_choose_chunk_size", "kvs_flash_decode_workspace_bytes",
           "kvs_flash_decode", "kvs_decode_step", "kvs_strerror", "kvs_flash_decode_static",
           "kvs_step_graph_create", "kvs_step_graph_launch", "kvs_step_graph_destroy",
           "kvs_set_schedule", "kvs_get_schedule", "kvs_schedule_for", "kvs_prepare",
           "kvs_decode_step_slots", "kvs_argmax", "kvs_prefill_attention",
           "kvs_prefill_workspace_bytes", "kvs_step_io_bytes", "kvs_decode_step_host",
           "kvs_set_wait_limit_ns", "kvs_step_io_layout", "kvs_decode_step_host_io",
           "kvs_step_graph_io_layout", "kvs_step_graph_create_host_io", "kvs_rope_scatter_paged",
           "kvs_rope_frequencies", "kvs_paged_attention_workspace_bytes", "kvs_paged_attention",
           "kvs_process_logits", "kvs_rope_scatter_paged_q8",
           "kvs_paged_attention_q8_workspace_bytes", "kvs_paged_attention_q8", "kvs_sample_logits")

# Positions of a kv head that share a scale in an 8-bit paged cache.
KVS_SCALE_BLOCK = 16

# Default bound on each pipeline wait of the kernels (kvs_set_wait_limit_ns).
KVS_WAIT_LIMIT_DEFAULT_NS = 2_000_000_000

# kvs_schedule values (kernel schedule of the attention entry points)
KVS_SCHEDULE_AUTO = 0
KVS_SCHEDULE_PERSISTENT = 1
KVS_SCHEDULE_CLUSTER = 2

# Size of the library's built-in scratch buffer used by kvs_flash_decode_static.
KVS_STATIC_WORKSPACE_BYTES = 32 * 1024 * 1024

_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_L = ctypes.c_int64
_F = ctypes.c_float
_D = ctypes.c_double


class KvsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {strerror(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m split_flash_decoding_kvcachescatter_gb300.build`")
            L = ctypes.CDLL(LIB_PATH)
            L.kvs_kv_scatter.restype = _I
            L.kvs_kv_scatter.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]
            L.kvs_choose_chunk_size.restype = _I
            L.kvs_choose_chunk_size.argtypes = [_I, _I, _I, _I, _I]
            L.kvs_flash_decode_workspace_bytes.restype = _SZ
            L.kvs_flash_decode_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
            L.kvs_flash_decode.restype = _I
            L.kvs_flash_decode.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                           _P, _SZ, _P, _P]
            L.kvs_decode_step.restype = _I
            L.kvs_decode_step.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                          _P, _SZ, _P, _P]
            L.kvs_step_io_bytes.restype = _SZ
            L.kvs_step_io_bytes.argtypes = [_I, _I, _I, _I]
            L.kvs_decode_step_host.restype = _I
            L.kvs_decode_step_host.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                               _I, _P, _SZ, _P, _SZ, _P, _P]
            L.kvs_flash_decode_static.restype = _I
            L.kvs_flash_decode_static.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                                  _P, _P]
            L.kvs_step_graph_create.restype = _I
            L.kvs_step_graph_create.argtypes = [_I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                                                _I, _I, _P, _SZ, _P, _P, _P]
            L.kvs_step_graph_launch.restype = _I
            L.kvs_step_graph_launch.argtypes = [_P, _P]
            L.kvs_step_graph_io_layout.restype = _I
            L.kvs_step_graph_io_layout.argtypes = [_I, _I, _I, _I, _I, _P]
            L.kvs_step_graph_create_host_io.restype = _I
            L.kvs_step_graph_create_host_io.argtypes = [_I, _P, _P, _SZ, _P, _P, _I, _I, _I, _I,
                                                        _I, _I, _P, _SZ, _P, _P, _P]
            L.kvs_step_graph_destroy.restype = _I
            L.kvs_step_graph_destroy.argtypes = [_P]
            L.kvs_decode_step_slots.restype = _I
            L.kvs_decode_step_slots.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _I,
                                                _I, _I, _I, _I, _P, _SZ, _P, _P]
            L.kvs_prefill_attention.restype = _I
            L.kvs_prefill_attention.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P,
                                                _P]
            L.kvs_prefill_workspace_bytes.restype = _SZ
            L.kvs_prefill_workspace_bytes.argtypes = [_I, _I, _I]
            L.kvs_argmax.restype = _I
            L.kvs_argmax.argtypes = [_P, _I, _I, _P, _P]
            L.kvs_set_schedule.restype = _I
            L.kvs_set_schedule.argtypes = [_I]
            L.kvs_get_schedule.restype = _I
            L.kvs_get_schedule.argtypes = []
            L.kvs_schedule_for.restype = _I
            L.kvs_schedule_for.argtypes = [_I, _I, _I, _I, _I]
            L.kvs_prepare.restype = _I
            L.kvs_prepare.argtypes = [_I, _I, _I]
            L.kvs_step_io_layout.restype = _I
            L.kvs_step_io_layout.argtypes = [_I, _I, _I, _I, ctypes.POINTER(_SZ)]
            L.kvs_decode_step_host_io.restype = _I
            L.kvs_decode_step_host_io.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ,
                                                  _P, _SZ, _P, _P]
            L.kvs_set_wait_limit_ns.restype = _I
            L.kvs_set_wait_limit_ns.argtypes = [ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint64)]
            L.kvs_rope_scatter_paged.restype = _I
            L.kvs_rope_scatter_paged.argtypes = [_P, _L, _P, _L, _P, _L, _P, _L, _P, _P, _P, _I,
                                                 _I, _I, _F, _P, _P]
            L.kvs_rope_frequencies.restype = _I
            L.kvs_rope_frequencies.argtypes = [_I, _D, _I, _D, _D, _D, _D, _P, _P]
            L.kvs_paged_attention_workspace_bytes.restype = _SZ
            L.kvs_paged_attention_workspace_bytes.argtypes = [_I, _I, _I, _I]
            L.kvs_paged_attention.restype = _I
            L.kvs_paged_attention.argtypes = [_P, _L, _P, _P, _P, _L, _I, _P, _SZ, _P, _P]
            L.kvs_process_logits.restype = _I
            L.kvs_process_logits.argtypes = [_P, _L, _P, _L, _I, _I, _I, _P, _P, _P, _P]
            L.kvs_rope_scatter_paged_q8.restype = _I
            L.kvs_rope_scatter_paged_q8.argtypes = [_P, _L, _P, _L, _P, _L, _P, _L, _I, _P, _P, _P,
                                                    _I, _I, _I, _F, _P, _P]
            L.kvs_paged_attention_q8_workspace_bytes.restype = _SZ
            L.kvs_paged_attention_q8_workspace_bytes.argtypes = [_I, _I, _I, _I]
            L.kvs_paged_attention_q8.restype = _I
            L.kvs_paged_attention_q8.argtypes = [_P, _L, _I, _P, _P, _P, _L, _I, _P, _SZ, _P, _P]
            L.kvs_sample_logits.restype = _I
            L.kvs_sample_logits.argtypes = [_P, _L, _I, _I, _I, _P, _P, _P, _P, _P, _L, _P]
            L.kvs_strerror.restype = ctypes.c_char_p
            L.kvs_strerror.argtypes = [_I]
            _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().kvs_strerror(int(status)).decode()


def _check(rc: int, where: str) -> None:
    if rc != KVS_OK:
        raise KvsError(rc, where)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _f32(t: torch.Tensor, name: str, ndim: int) -> int:
    if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous() and t.dim() == ndim):
        raise TypeError(f"{name}: need a contiguous float32 CUDA tensor with {ndim} dims, got "
                        f"{tuple(t.shape)} {t.dtype} {t.device}")
    return t.data_ptr()


def _i32(t: torch.Tensor, name: str) -> int:
    if not (t.is_cuda and t.dtype == torch.int32 and t.is_contiguous() and t.dim() == 1):
        raise TypeError(f"{name}: need a contiguous int32 CUDA vector")
    return t.data_ptr()


def _status_ptr(d_status) -> int:
    if d_status is None:
        return 0
    if not (d_status.is_cuda and d_status.dtype == torch.int32):
        raise TypeError("d_status: need an int32 CUDA tensor")
    return d_status.data_ptr()


def kvs_kv_scatter(k_rows, v_rows, positions, k_cache, v_cache, d_status=None, stream=None):
    """Scatter k_rows/v_rows [M,Hkv,D] into caches [M,Hkv,Lmax,D] at positions [M]."""
    M, Hkv, Lmax, D = k_cache.shape
    if tuple(v_cache.shape) != (M, Hkv, Lmax, D) or tuple(k_rows.shape) != (M, Hkv, D) or \
            tuple(v_rows.shape) != (M, Hkv, D) or positions.numel() != M:
        raise ValueError("kvs_kv_scatter: inconsistent shapes")
    rc = lib().kvs_kv_scatter(_f32(k_rows, "k_rows", 3), _f32(v_rows, "v_rows", 3),
                              _i32(positions, "positions"), _f32(k_cache, "k_cache", 4),
                              _f32(v_cache, "v_cache", 4), M, Hkv, D, Lmax,
                              _status_ptr(d_status), _stream(stream))
    _check(rc, "kvs_kv_scatter")


def prefill_workspace(H, S, D, device=None):
    """A device byte buffer large enough for kvs_prefill_attention (allocated by torch)."""
    n = int(lib().kvs_prefill_workspace_bytes(H, S, D))
    if n == 0:
        raise KvsError(KVS_ERR_DIMS, "kvs_prefill_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def kvs_prefill_attention(q, k, v, out, causal=True, workspace=None, d_status=None, stream=None):
    """Tensor-core attention over whole sequences: q, k, v, out [H, S, D] float32 (CUDA)."""
    H, S, D = q.shape
    for name, t in (("k", k), ("v", v), ("out", out)):
        if tuple(t.shape) != (H, S, D):
            raise ValueError(f"kvs_prefill_attention: {name} must be [H, S, D] like q")
    if workspace is None:
        raise ValueError("kvs_prefill_attention: pass a workspace (see binding.prefill_workspace)")
    _check(lib().kvs_prefill_attention(_f32(q, "q", 3), _f32(k, "k", 3), _f32(v, "v", 3),
                                       _f32(out, "out", 3), H, S, D, 1 if causal else 0,
                                       workspace.data_ptr(),
                                       workspace.numel() * workspace.element_size(),
                                       _status_ptr(d_status), _stream(stream)),
           "kvs_prefill_attention")
    return out


def kvs_argmax(logits, token_ids=None, stream=None):
    """Greedy token of each row of logits [M, V] (float32, CUDA): int32 [M] on the device."""
    if not (logits.is_cuda and logits.dtype == torch.float32 and logits.dim() == 2 and
            logits.stride(1) == 1 and logits.stride(0) == logits.shape[1]):
        raise TypeError("logits: need a contiguous float32 CUDA matrix [M, V]")
    M, V = logits.shape
    if token_ids is None:
        token_ids = torch.empty(M, dtype=torch.int32, device=logits.device)
    _check(lib().kvs_argmax(logits.data_ptr(), M, V, _i32(token_ids, "token_ids"),
                            _stream(stream)), "kvs_argmax")
    return token_ids


def kvs_set_schedule(schedule: int) -> int:
    """Set the process-wide kernel schedule (KVS_SCHEDULE_*); returns the previous one."""
    prev = lib().kvs_set_schedule(int(schedule))
    if prev < 0:
        raise KvsError(-prev, "kvs_set_schedule")
    return prev


def kvs_get_schedule() -> int:
    return int(lib().kvs_get_schedule())


def kvs_schedule_for(M, num_heads, num_kv_heads, head_dim, max_len) -> int:
    """KVS_SCHEDULE_PERSISTENT or KVS_SCHEDULE_CLUSTER: the kernel such a call would run."""
    r = lib().kvs_schedule_for(M, num_heads, num_kv_heads, head_dim, max_len)
    if r < 0:
        raise KvsError(-r, "kvs_schedule_for")
    return r


def kvs_set_wait_limit_ns(ns: int) -> int:
    """Set the bound on each pipeline wait of the kernels on the current
    device (0 .. KVS_WAIT_LIMIT_DEFAULT_NS); returns the previous bound."""
    prev = ctypes.c_uint64(0)
    _check(lib().kvs_set_wait_limit_ns(int(ns), ctypes.byref(prev)), "kvs_set_wait_limit_ns")
    return int(prev.value)


def kvs_prepare(num_heads, num_kv_heads, head_dim) -> None:
    """Set up both attention kernels for this shape on the current device."""
    _check(lib().kvs_prepare(num_heads, num_kv_heads, head_dim), "kvs_prepare")


def kvs_choose_chunk_size(M, num_kv_heads, head_dim, max_len, num_sms=0) -> int:
    c = lib().kvs_choose_chunk_size(M, num_kv_heads, head_dim, max_len, num_sms)
    if c <= 0:
        raise KvsError(-c, "kvs_choose_chunk_size")
    return c


def kvs_flash_decode_workspace_bytes(M, num_heads, num_kv_heads, head_dim, max_len,
                                     chunk_size) -> int:
    return int(lib().kvs_flash_decode_workspace_bytes(M, num_heads, num_kv_heads, head_dim,
                                                      max_len, chunk_size))


def workspace(M, num_heads, num_kv_heads, head_dim, max_len, chunk_size, device=None):
    """A device byte buffer large enough for kvs_flash_decode (allocated by torch)."""
    n = kvs_flash_decode_workspace_bytes(M, num_heads, num_kv_heads, head_dim, max_len,
                                         chunk_size)
    if n == 0 and M > 0:
        raise KvsError(KVS_ERR_DIMS, "kvs_flash_decode_workspace_bytes")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def _attn_shapes(q, k_cache):
    M, H, D = q.shape
    M2, Hkv, Lmax, D2 = k_cache.shape
    if M2 != M or D2 != D:
        raise ValueError("q and k_cache disagree on M or head_dim")
    return M, H, Hkv, D, Lmax


def kvs_flash_decode(q, k_cache, v_cache, positions, out, chunk_size=0, workspace=None,
                     d_status=None, stream=None):
    """out[M,H,D] = split-K softmax attention of q over cache rows 0..positions[i]."""
    M, H, Hkv, D, Lmax = _attn_shapes(q, k_cache)
    if workspace is None:
        raise ValueError("kvs_flash_decode: pass a workspace (see binding.workspace)")
    rc = lib().kvs_flash_decode(_f32(q, "q", 3), _f32(k_cache, "k_cache", 4),
                                _f32(v_cache, "v_cache", 4), _i32(positions, "positions"),
                                _f32(out, "out", 3), M, H, Hkv, D, Lmax, int(chunk_size),
                                workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _status_ptr(d_status), _stream(stream))
    _check(rc, "kvs_flash_decode")


def kvs_decode_step(q, k_rows, v_rows, positions, k_cache, v_cache, out, chunk_size=0,
                    workspace=None, d_status=None, stream=None):
    """kvs_kv_scatter + kvs_flash_decode of one layer's decode step, in one launch."""
    M, H, Hkv, D, Lmax = _attn_shapes(q, k_cache)
    if workspace is None:
        raise ValueError("kvs_decode_step: pass a workspace (see binding.workspace)")
    if tuple(k_rows.shape) != (M, Hkv, D) or tuple(v_rows.shape) != (M, Hkv, D) or \
            tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("kvs_decode_step: inconsistent shapes")
    rc = lib().kvs_decode_step(_f32(q, "q", 3), _f32(k_rows, "k_rows", 3),
                               _f32(v_rows, "v_rows", 3), _i32(positions, "positions"),
                               _f32(k_cache, "k_cache", 4), _f32(v_cache, "v_cache", 4),
                               _f32(out, "out", 3), M, H, Hkv, D, Lmax, int(chunk_size),
                               workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                               _status_ptr(d_status), _stream(stream))
    _check(rc, "kvs_decode_step")


def step_io(M, num_heads, num_kv_heads, head_dim, device=None):
    """A device byte buffer large enough for kvs_decode_step_host's copies."""
    n = int(lib().kvs_step_io_bytes(M, num_heads, num_kv_heads, head_dim))
    if n == 0:
        raise KvsError(KVS_ERR_DIMS, "kvs_step_io_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _host(t: torch.Tensor, name: str, dtype, shape) -> int:
    if t.is_cuda or t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise TypeError(f"{name}: need a contiguous {dtype} CPU tensor of shape {tuple(shape)}, "
                        f"got {tuple(t.shape)} {t.dtype} {t.device}")
    return t.data_ptr()


def kvs_decode_step_host(q, k_rows, v_rows, positions, k_cache, v_cache, out, chunk_size=0,
                         workspace=None, io=None, d_status=None, stream=None):
    """kvs_decode_step with q, k_rows, v_rows, positions and out in host memory
    (CPU tensors, pinned for asynchronous copies): the copies in, the fused
    step and the copy of out back, enqueued by one library call.  out is valid
    after the stream is synchronised."""
    M, Hkv, Lmax, D = k_cache.shape
    H = q.shape[1] if q.dim() == 3 else -1
    if workspace is None or io is None:
        raise ValueError("kvs_decode_step_host: pass a workspace and an io buffer "
                         "(see binding.workspace, binding.step_io)")
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("kvs_decode_step_host: inconsistent cache shapes")
    rc = lib().kvs_decode_step_host(
        _host(q, "q", torch.float32, (M, H, D)), _host(k_rows, "k_rows", torch.float32, (M, Hkv, D)),
        _host(v_rows, "v_rows", torch.float32, (M, Hkv, D)),
        _host(positions, "positions", torch.int32, (M,)),
        _f32(k_cache, "k_cache", 4), _f32(v_cache, "v_cache", 4),
        _host(out, "out", torch.float32, (M, H, D)), M, H, Hkv, D, Lmax, int(chunk_size),
        io.data_ptr(), io.numel() * io.element_size(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _status_ptr(d_status), _stream(stream))
    _check(rc, "kvs_decode_step_host")


def kvs_step_io_layout(M, num_heads, num_kv_heads, head_dim):
    """Byte offsets of q, k_rows, v_rows, positions, out and the total size
    of an io buffer (device, or the host buffer of kvs_decode_step_host_io)."""
    off = (_SZ * 6)()
    _check(lib().kvs_step_io_layout(M, num_heads, num_kv_heads, head_dim, off),
           "kvs_step_io_layout")
    return tuple(int(x) for x in off)


class HostIo:
    """A host buffer with the io layout, and views of its arrays: fill q,
    k_rows, v_rows and positions, call kvs_decode_step_host_io, and read out
    once the stream has passed the call.  Pinned by default (the library then
    moves it with its copy kernel); pinned=False gives pageable memory (moved
    by copy engines, the host waiting for them)."""

    def __init__(self, M, num_heads, num_kv_heads, head_dim, pinned=True):
        oq, ok, ov, op, oo, total = kvs_step_io_layout(M, num_heads, num_kv_heads, head_dim)
        self.shape = (M, num_heads, num_kv_heads, head_dim)
        self.buf = torch.empty(total, dtype=torch.uint8, pin_memory=pinned)
        f = lambda off, n, dt: self.buf[off:off + n * 4].view(dt)
        self.q = f(oq, M * num_heads * head_dim, torch.float32).view(M, num_heads, head_dim)
        self.k_rows = f(ok, M * num_kv_heads * head_dim, torch.float32).view(
            M, num_kv_heads, head_dim)
        self.v_rows = f(ov, M * num_kv_heads * head_dim, torch.float32).view(
            M, num_kv_heads, head_dim)
        self.positions = f(op, M, torch.int32)
        self.out = f(oo, M * num_heads * head_dim, torch.float32).view(M, num_heads, head_dim)
        self.in_bytes = op + 4 * M          # what one step copies to the device
        self.out_bytes = M * num_heads * head_dim * 4  # and back


def kvs_decode_step_host_io(host_io, k_cache, v_cache, chunk_size=0, workspace=None, io=None,
                            d_status=None, stream=None):
    """kvs_decode_step with the step's inputs and result in one pinned host
    buffer (a HostIo): one copy in, the fused step, one copy out."""
    M, Hkv, Lmax, D = k_cache.shape
    if not isinstance(host_io, HostIo):
        raise TypeError("host_io: need a binding.HostIo")
    Mh, H, Hkvh, Dh = host_io.shape
    if (Mh, Hkvh, Dh) != (M, Hkv, D) or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("kvs_decode_step_host_io: inconsistent shapes")
    if workspace is None or io is None:
        raise ValueError("kvs_decode_step_host_io: pass a workspace and an io buffer")
    rc = lib().kvs_decode_step_host_io(
        host_io.buf.data_ptr(), _f32(k_cache, "k_cache", 4), _f32(v_cache, "v_cache", 4), M, H,
        Hkv, D, Lmax, int(chunk_size), io.data_ptr(), io.numel() * io.element_size(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _status_ptr(d_status), _stream(stream))
    _check(rc, "kvs_decode_step_host_io")


def kvs_step_graph_io_layout(layers, M, num_heads, num_kv_heads, head_dim):
    """Offsets of kvs_step_graph_io_layout: a list of 4 * layers + 2 ints."""
    off = (ctypes.c_size_t * (4 * layers + 2))()
    _check(lib().kvs_step_graph_io_layout(layers, M, num_heads, num_kv_heads, head_dim, off),
           "kvs_step_graph_io_layout")
    return list(off)


class HostStepIo:
    """A pinned host buffer with the layout of kvs_step_graph_io_layout and
    views of its arrays: q[l], k_rows[l], v_rows[l], out[l] per layer and the
    shared positions.  Fill the inputs, launch the host-io step graph, read
    the outs once the stream has passed the launch."""

    def __init__(self, layers, M, num_heads, num_kv_heads, head_dim):
        off = kvs_step_graph_io_layout(layers, M, num_heads, num_kv_heads, head_dim)
        self.layers, self.shape = layers, (M, num_heads, num_kv_heads, head_dim)
        self.total = off[4 * layers + 1]
        self.buf = torch.empty(self.total, dtype=torch.uint8, pin_memory=True)
        f = lambda o, n, dt: self.buf[o:o + n * 4].view(dt)
        qn, kn = M * num_heads * head_dim, M * num_kv_heads * head_dim
        self.q = [f(off[3 * l], qn, torch.float32).view(M, num_heads, head_dim)
                  for l in range(layers)]
        self.k_rows = [f(off[3 * l + 1], kn, torch.float32).view(M, num_kv_heads, head_dim)
                       for l in range(layers)]
        self.v_rows = [f(off[3 * l + 2], kn, torch.float32).view(M, num_kv_heads, head_dim)
                       for l in range(layers)]
        self.positions = f(off[3 * layers], M, torch.int32)
        self.out = [f(off[3 * layers + 1 + l], qn, torch.float32).view(M, num_heads, head_dim)
                    for l in range(layers)]
        self.in_bytes = off[3 * layers + 1]          # one copy to the device a step
        self.out_bytes = self.total - self.in_bytes  # and one back


def kvs_step_graph_create_host_io(host_io, k_cache, v_cache, chunk_size=0, workspace=None,
                                  io=None, d_status=None, stream=None):
    """A step graph over one pinned host buffer (a HostStepIo): one copy of
    every layer's inputs in, the layers, one copy of every layer's out back."""
    if not isinstance(host_io, HostStepIo):
        raise TypeError("host_io: need a binding.HostStepIo")
    layers = host_io.layers
    if not (len(k_cache) == len(v_cache) == layers):
        raise ValueError("kvs_step_graph_create_host_io: one cache per layer")
    if workspace is None or io is None:
        raise ValueError("kvs_step_graph_create_host_io: pass a workspace and an io buffer")
    M, Hkv, Lmax, D = k_cache[0].shape
    Mh, H, Hkvh, Dh = host_io.shape
    if (Mh, Hkvh, Dh) != (M, Hkv, D):
        raise ValueError("kvs_step_graph_create_host_io: inconsistent shapes")
    arr = lambda ts, name: (ctypes.c_void_p * layers)(*[_f32(t, name, 4) for t in ts])
    s = torch.cuda.Stream() if stream is None else stream
    handle = ctypes.c_void_p()
    rc = lib().kvs_step_graph_create_host_io(
        layers, host_io.buf.data_ptr(), io.data_ptr(), io.numel() * io.element_size(),
        arr(k_cache, "k_cache"), arr(v_cache, "v_cache"), M, H, Hkv, D, Lmax, int(chunk_size),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _status_ptr(d_status), _stream(s), ctypes.byref(handle))
    _check(rc, "kvs_step_graph_create_host_io")
    return StepGraph(handle, (host_io, io, k_cache, v_cache, workspace))


def kvs_decode_step_slots(q, k_rows, v_rows, positions, slots, done, k_pool, v_pool, out,
                          chunk_size=0, workspace=None, d_status=None, stream=None):
    """Decode step over a cache pool [S, Hkv, Lmax, D]: sequence i uses slot
    slots[i] (int32 [M], or None for slot i); done (uint8 [M] or None) marks
    finished sequences, which are scattered but not attended (their out rows
    are left as they are).  k_rows and v_rows both None: attention only."""
    M, H, D = q.shape
    S, Hkv, Lmax, D2 = k_pool.shape
    if D2 != D or tuple(v_pool.shape) != tuple(k_pool.shape) or tuple(out.shape) != (M, H, D):
        raise ValueError("kvs_decode_step_slots: inconsistent shapes")
    if workspace is None:
        raise ValueError("kvs_decode_step_slots: pass a workspace (see binding.workspace)")
    if (k_rows is None) != (v_rows is None):
        raise ValueError("kvs_decode_step_slots: pass both k_rows and v_rows, or neither")
    kr = 0 if k_rows is None else _f32(k_rows, "k_rows", 3)
    vr = 0 if v_rows is None else _f32(v_rows, "v_rows", 3)
    if k_rows is not None and (tuple(k_rows.shape) != (M, Hkv, D) or
                               tuple(v_rows.shape) != (M, Hkv, D)):
        raise ValueError("kvs_decode_step_slots: k_rows / v_rows must be [M, Hkv, D]")
    sl = 0 if slots is None else _i32(slots, "slots")
    if slots is not None and slots.numel() != M:
        raise ValueError("kvs_decode_step_slots: slots must have M entries")
    dn = 0
    if done is not None:
        if not (done.is_cuda and done.dtype == torch.uint8 and done.is_contiguous() and
                done.numel() == M):
            raise TypeError("done: need a contiguous uint8 CUDA vector of M entries")
        dn = done.data_ptr()
    rc = lib().kvs_decode_step_slots(_f32(q, "q", 3), kr, vr, _i32(positions, "positions"), sl,
                                     dn, _f32(k_pool, "k_pool", 4), _f32(v_pool, "v_pool", 4), S,
                                     _f32(out, "out", 3), M, H, Hkv, D, Lmax, int(chunk_size),
                                     workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(),
                                     _status_ptr(d_status), _stream(stream))
    _check(rc, "kvs_decode_step_slots")


def kvs_flash_decode_static(q, k_cache, v_cache, positions, out, chunk_size=0, d_status=None,
                            stream=None):
    """kvs_flash_decode without a workspace argument: the partials go to the
    library's built-in buffer (for callers that cannot allocate device memory;
    calls that may overlap on the GPU must be ordered, see the C header)."""
    M, H, Hkv, D, Lmax = _attn_shapes(q, k_cache)
    rc = lib().kvs_flash_decode_static(_f32(q, "q", 3), _f32(k_cache, "k_cache", 4),
                                       _f32(v_cache, "v_cache", 4),
                                       _i32(positions, "positions"), _f32(out, "out", 3), M, H,
                                       Hkv, D, Lmax, int(chunk_size), _status_ptr(d_status),
                                       _stream(stream))
    _check(rc, "kvs_flash_decode_static")


class StepGraph:
    """Handle of kvs_step_graph_create: a whole multi-layer decode step as one
    CUDA graph over fixed buffers (update their contents, not their
    addresses, between launches)."""

    def __init__(self, handle, keep):
        self._h = handle
        self._keep = keep  # the captured tensors must outlive the graph

    def launch(self, stream=None):
        _check(lib().kvs_step_graph_launch(self._h, _stream(stream)), "kvs_step_graph_launch")

    def destroy(self):
        if self._h:
            lib().kvs_step_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def kvs_step_graph_create(q, k_rows, v_rows, positions, k_cache, v_cache, out, chunk_size=0,
                          workspace=None, d_status=None, stream=None):
    """Capture one kvs_decode_step per layer (lists of per-layer tensors)."""
    layers = len(q)
    if not (len(k_rows) == len(v_rows) == len(k_cache) == len(v_cache) == len(out) == layers):
        raise ValueError("kvs_step_graph_create: one tensor per layer in every list")
    if workspace is None:
        raise ValueError("kvs_step_graph_create: pass a workspace")
    M, H, Hkv, D, Lmax = _attn_shapes(q[0], k_cache[0])
    arr = lambda ts, name, nd: (ctypes.c_void_p * layers)(*[_f32(t, name, nd) for t in ts])
    s = torch.cuda.Stream() if stream is None else stream
    handle = ctypes.c_void_p()
    rc = lib().kvs_step_graph_create(
        layers, arr(q, "q", 3), arr(k_rows, "k_rows", 3), arr(v_rows, "v_rows", 3),
        _i32(positions, "positions"), arr(k_cache, "k_cache", 4), arr(v_cache, "v_cache", 4),
        arr(out, "out", 3), M, H, Hkv, D, Lmax, int(chunk_size), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _status_ptr(d_status), _stream(s),
        ctypes.byref(handle))
    _check(rc, "kvs_step_graph_create")
    return StepGraph(handle, (q, k_rows, v_rows, positions, k_cache, v_cache, out, workspace))


class _PagedCacheStruct(ctypes.Structure):
    _fields_ = [("k_pages", _P), ("v_pages", _P), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class _PagedCacheQ8Struct(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k_pages", "v_pages", "k_scales", "v_scales")] + \
               [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "num_kv_heads", "head_dim")]


class _PagedBatchStruct(ctypes.Structure):
    _fields_ = [("positions", _P), ("row_offsets", _P), ("page_table", _P),
                ("num_seqs", ctypes.c_int32), ("num_rows", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class _LogitRulesStruct(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("history", "history_offsets", "prompt_lens", "repetition",
                                  "presence", "frequency", "bias_ids", "bias_values",
                                  "bias_offsets", "mask", "mask_rows")] + \
               [(n, ctypes.c_int32) for n in ("history_len", "bias_len", "mask_count")]


class PagedCache:
    """A paged KV cache, checked once: k_pages and v_pages [num_pages, Hkv, page_size, D]
    (float32, float16 or bfloat16, contiguous, CUDA)."""

    def __init__(self, k_pages, v_pages):
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not (t.is_cuda and t.dtype in _DTYPES and t.dim() == 4 and t.is_contiguous()):
                raise TypeError(f"{name}: need a contiguous CUDA tensor [num_pages, Hkv, page_size, "
                                f"D] of float32, float16 or bfloat16, got {tuple(t.shape)} "
                                f"{t.dtype} {t.device}")
        if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype or \
                k_pages.device != v_pages.device:
            raise ValueError("PagedCache: k_pages and v_pages differ in shape, type or device")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.dtype, self.device_index = k_pages.dtype, k_pages.get_device()
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = k_pages.shape
        self._struct = _PagedCacheStruct(k_pages.data_ptr(), v_pages.data_ptr(), self.num_pages,
                                         self.page_size, self.num_kv_heads, self.head_dim,
                                         _DTYPES[k_pages.dtype])
        self._addr = ctypes.addressof(self._struct)
        self._call = lib().kvs_paged_attention, lib().kvs_rope_scatter_paged


class PagedCacheQ8:
    """A paged KV cache in 8 bits, checked once: k_pages and v_pages [num_pages, Hkv, page_size, D]
    (float8_e4m3fn), k_scales and v_scales [num_pages, Hkv, page_size / 16] (float32); contiguous,
    CUDA.  An element is its block's scale times the stored number."""

    def __init__(self, k_pages, v_pages, k_scales, v_scales):
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not (t.is_cuda and t.dtype is torch.float8_e4m3fn and t.dim() == 4 and
                    t.is_contiguous()):
                raise TypeError(f"{name}: need a contiguous CUDA tensor [num_pages, Hkv, page_size, "
                                f"D] of float8_e4m3fn, got {tuple(t.shape)} {t.dtype} {t.device}")
        if k_pages.shape != v_pages.shape or k_pages.device != v_pages.device:
            raise ValueError("PagedCacheQ8: k_pages and v_pages differ in shape or device")
        shape = (*k_pages.shape[:2], k_pages.shape[2] // KVS_SCALE_BLOCK)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if not (t.dtype is torch.float32 and t.shape == shape and t.is_contiguous() and
                    t.device == k_pages.device):
                raise TypeError(f"{name}: need a contiguous float32 tensor {list(shape)} on "
                                f"{k_pages.device}, got {tuple(t.shape)} {t.dtype} {t.device}")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.k_scales, self.v_scales = k_scales, v_scales
        self.device_index = k_pages.get_device()
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = k_pages.shape
        self._struct = _PagedCacheQ8Struct(k_pages.data_ptr(), v_pages.data_ptr(),
                                           k_scales.data_ptr(), v_scales.data_ptr(), self.num_pages,
                                           self.page_size, self.num_kv_heads, self.head_dim)
        self._addr = ctypes.addressof(self._struct)
        self._call = lib().kvs_paged_attention_q8, lib().kvs_rope_scatter_paged_q8


class PagedBatch:
    """A ragged batch over a paged cache, checked once: positions [M], row_offsets [M + 1] and
    page_table [M, max_pages] (int32, contiguous, CUDA).  Update the tensors' contents between
    calls, not their addresses; num_rows (rows of q, k, v and out) and max_new (the largest
    number of new tokens of a sequence) are the caller's, since the offsets are on the device."""

    def __init__(self, positions, row_offsets, page_table, num_rows, max_new):
        p, o = _i32(positions, "positions"), _i32(row_offsets, "row_offsets")
        if not (page_table.is_cuda and page_table.dtype == torch.int32 and
                page_table.dim() == 2 and page_table.is_contiguous()):
            raise TypeError("page_table: need a contiguous int32 CUDA matrix [M, max_pages]")
        M = positions.numel()
        if row_offsets.numel() != M + 1 or page_table.shape[0] != M:
            raise ValueError("PagedBatch: positions [M], row_offsets [M + 1] and page_table "
                             "[M, max_pages] disagree on M")
        if not positions.get_device() == row_offsets.get_device() == page_table.get_device():
            raise ValueError("PagedBatch: tensors on different devices")
        self.positions, self.row_offsets, self.page_table = positions, row_offsets, page_table
        self.num_seqs, self.num_rows, self.max_new = M, int(num_rows), int(max_new)
        self.device_index = positions.get_device()
        self._struct = _PagedBatchStruct(p, o, page_table.data_ptr(), M, self.num_rows,
                                         self.max_new, page_table.shape[1])
        self._addr = ctypes.addressof(self._struct)


# The paged-cache and logit calls are a few microseconds of GPU work in a
# decode step, so their checks are written to cost little: handles are
# checked once, tensors by as few attribute reads as say it.
_get_device = torch._C._cuda_getDevice
_get_stream = torch._C._cuda_getCurrentRawStream


def _call_device(dev: int, where: str) -> None:
    """The call's tensors (on device dev) must be on the current device."""
    if dev < 0 or dev != _get_device():
        raise ValueError(f"{where}: the tensors are on device {dev}, which is not the current one")


def _bad_rows(where: str, dtype, dev: int, **tensors) -> None:
    """Raises for the first (tensor, shape) that is not [rows, heads, D] as the call needs it."""
    for name, (t, shape) in tensors.items():
        if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
            raise TypeError(f"{where}: {name}: need a {dtype} tensor {list(shape)} on device {dev}, "
                            f"got {tuple(t.shape)} {t.dtype} {t.device}")
        s = t.stride()
        if s[2] != 1 or (s[1] != shape[2] and shape[1] > 1):
            raise TypeError(f"{where}: {name}: the [heads, D] rows must be contiguous, got strides {s}")
    raise AssertionError(where)


def kvs_rope_frequencies(rot_dim, base=10000.0, kind=KVS_ROPE_PLAIN, factor=1.0, original_len=0.0,
                         slow=1.0, fast=32.0, device=None):
    """(inv_freq, scale): the frequency table of kvs_rope_scatter_paged (float32 [rot_dim / 2] on
    the device) and the factor it goes with, for a length-scaling rule KVS_ROPE_*."""
    table = torch.empty(max(rot_dim // 2, 1), dtype=torch.float32)
    scale = ctypes.c_float(1.0)
    _check(lib().kvs_rope_frequencies(int(rot_dim), float(base), int(kind), float(factor),
                                      float(original_len), float(slow), float(fast),
                                      table.data_ptr(), ctypes.addressof(scale)),
           "kvs_rope_frequencies")
    return table.to(device or "cuda"), scale.value


def kvs_rope_scatter_paged(q, k, v, q_out, cache, batch, inv_freq, interleaved=False, scale=1.0,
                           d_status=None, stream=None):
    """Rotary positions on q [num_rows, H, D] and k [num_rows, Hkv, D] of a PagedBatch: rotated q
    to q_out (q itself is fine), rotated k and plain v into the pages of a PagedCache.  Rows may
    be strided (column blocks of one matrix).  The head's first 2 * inv_freq.numel() elements
    turn, the rest is copied."""
    dev, dt, N, D, Hkv = (cache.device_index, cache.dtype, batch.num_rows, cache.head_dim,
                          cache.num_kv_heads)
    if dev != _get_device() or batch.device_index != dev:
        raise ValueError("kvs_rope_scatter_paged: cache and batch must be on the current device")
    H = q.shape[1] if q.dim() == 3 else -1
    if inv_freq.dtype is not torch.float32 or inv_freq.get_device() != dev or \
            inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq: need a contiguous float32 vector on the tensors' device")
    of_q, of_kv = (N, H, D), (N, Hkv, D)
    if not (q.dtype is k.dtype is v.dtype is q_out.dtype is dt and
            q.get_device() == k.get_device() == v.get_device() == q_out.get_device() == dev and
            q.shape == of_q == q_out.shape and k.shape == of_kv == v.shape):
        _bad_rows("kvs_rope_scatter_paged", dt, dev, q=(q, of_q), k=(k, of_kv), v=(v, of_kv),
                  q_out=(q_out, of_q))
    qs, ks, vs, os_ = q.stride(), k.stride(), v.stride(), q_out.stride()
    if not (qs[2] == ks[2] == vs[2] == os_[2] == 1 and (qs[1] == os_[1] == D or H == 1) and
            (ks[1] == vs[1] == D or Hkv == 1)):
        _bad_rows("kvs_rope_scatter_paged", dt, dev, q=(q, of_q), k=(k, of_kv), v=(v, of_kv),
                  q_out=(q_out, of_q))
    if N > 1:
        qs, ks, vs, os_ = qs[0], ks[0], vs[0], os_[0]
    else:  # (the stride of a single row says nothing)
        qs = os_ = H * D
        ks = vs = Hkv * D
    rc = cache._call[1](q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, q_out.data_ptr(), os_,
                        cache._addr, batch._addr, inv_freq.data_ptr(), H, 2 * inv_freq.numel(),
                        1 if interleaved else 0, scale,
                        0 if d_status is None else _status_ptr(d_status),
                        _get_stream(dev) if stream is None else _stream(stream))
    if rc != KVS_OK:
        raise KvsError(rc, "kvs_rope_scatter_paged")
    return q_out


def paged_attention_workspace(cache, batch, num_heads, device=None):
    """A device byte buffer large enough for kvs_paged_attention (allocated by torch)."""
    n = int(lib().kvs_paged_attention_workspace_bytes(num_heads, cache.num_kv_heads,
                                                      cache.head_dim, batch.max_new))
    if n == 0:
        raise KvsError(KVS_ERR_DIMS, "kvs_paged_attention_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or cache.k_pages.device)


def kvs_paged_attention(q, cache, batch, out, workspace=None, d_status=None, stream=None):
    """out [num_rows, H, D] = attention of every new token of a PagedBatch over its sequence's
    pages, rows 0 .. its own position."""
    dev, dt, N, D = cache.device_index, cache.dtype, batch.num_rows, cache.head_dim
    if dev != _get_device() or batch.device_index != dev:
        raise ValueError("kvs_paged_attention: cache and batch must be on the current device")
    if workspace is None:
        raise ValueError("kvs_paged_attention: pass a workspace (see "
                         "binding.paged_attention_workspace)")
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise TypeError("kvs_paged_attention: the workspace must be a contiguous tensor on the "
                        "tensors' device")
    H = q.shape[1] if q.dim() == 3 else -1
    shape = (N, H, D)
    if not (q.dtype is out.dtype is dt and q.get_device() == out.get_device() == dev and
            q.shape == shape == out.shape):
        _bad_rows("kvs_paged_attention", dt, dev, q=(q, shape), out=(out, shape))
    qs, os_ = q.stride(), out.stride()
    if not (qs[2] == os_[2] == 1 and (qs[1] == os_[1] == D or H == 1)):
        _bad_rows("kvs_paged_attention", dt, dev, q=(q, shape), out=(out, shape))
    if N > 1:
        qs, os_ = qs[0], os_[0]
    else:  # (the stride of a single row says nothing)
        qs = os_ = H * D
    qp, op = q.data_ptr(), out.data_ptr()
    if qp == op and N > 0:
        raise ValueError("kvs_paged_attention: out must not overlap q")
    rc = cache._call[0](qp, qs, cache._addr, batch._addr, op, os_, H,
                        workspace.data_ptr(), workspace.nbytes,
                        0 if d_status is None else _status_ptr(d_status),
                        _get_stream(dev) if stream is None else _stream(stream))
    if rc != KVS_OK:
        raise KvsError(rc, "kvs_paged_attention")
    return out


def _q8_rows(where, q, cache, batch):
    """(dtype, kvs_dtype, device, heads) of a call's q over a PagedCacheQ8."""
    dev = cache.device_index
    if dev != _get_device() or batch.device_index != dev:
        raise ValueError(f"{where}: cache and batch must be on the current device")
    dt = q.dtype
    kd = _DTYPES.get(dt)
    if kd is None:
        raise TypeError(f"{where}: q: need float32, float16 or bfloat16, got {dt}")
    return dt, kd, dev, q.shape[1] if q.dim() == 3 else -1


def kvs_rope_scatter_paged_q8(q, k, v, q_out, cache, batch, inv_freq, interleaved=False, scale=1.0,
                              d_status=None, stream=None):
    """kvs_rope_scatter_paged into a PagedCacheQ8: rotated q to q_out, rotated k and plain v rounded
    to 8 bits into the pages, with a power of two as the scale of each 16 positions of a kv head.
    q, k, v and q_out have one type (float32, float16 or bfloat16)."""
    where = "kvs_rope_scatter_paged_q8"
    dt, kd, dev, H = _q8_rows(where, q, cache, batch)
    N, D, Hkv = batch.num_rows, cache.head_dim, cache.num_kv_heads
    if inv_freq.dtype is not torch.float32 or inv_freq.get_device() != dev or \
            inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq: need a contiguous float32 vector on the tensors' device")
    of_q, of_kv = (N, H, D), (N, Hkv, D)
    qs, ks, vs, os_ = q.stride(), k.stride(), v.stride(), q_out.stride()
    if not (k.dtype is v.dtype is q_out.dtype is dt and
            q.get_device() == k.get_device() == v.get_device() == q_out.get_device() == dev and
            q.shape == of_q == q_out.shape and k.shape == of_kv == v.shape and
            qs[2] == ks[2] == vs[2] == os_[2] == 1 and (qs[1] == os_[1] == D or H == 1) and
            (ks[1] == vs[1] == D or Hkv == 1)):
        _bad_rows(where, dt, dev, q=(q, of_q), k=(k, of_kv), v=(v, of_kv), q_out=(q_out, of_q))
    if N > 1:
        qs, ks, vs, os_ = qs[0], ks[0], vs[0], os_[0]
    else:  # (the stride of a single row says nothing)
        qs = os_ = H * D
        ks = vs = Hkv * D
    rc = cache._call[1](q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, q_out.data_ptr(), os_,
                        kd, cache._addr, batch._addr, inv_freq.data_ptr(), H, 2 * inv_freq.numel(),
                        1 if interleaved else 0, scale,
                        0 if d_status is None else _status_ptr(d_status),
                        _get_stream(dev) if stream is None else _stream(stream))
    if rc != KVS_OK:
        raise KvsError(rc, where)
    return q_out


def paged_attention_q8_workspace(cache, batch, num_heads, device=None):
    """A device byte buffer large enough for kvs_paged_attention_q8 (allocated by torch)."""
    n = int(lib().kvs_paged_attention_q8_workspace_bytes(num_heads, cache.num_kv_heads,
                                                         cache.head_dim, batch.max_new))
    if n == 0:
        raise KvsError(KVS_ERR_DIMS, "kvs_paged_attention_q8_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or cache.k_pages.device)


def kvs_paged_attention_q8(q, cache, batch, out, workspace=None, d_status=None, stream=None):
    """kvs_paged_attention over a PagedCacheQ8; q and out have one type (float32, float16 or
    bfloat16)."""
    where = "kvs_paged_attention_q8"
    dt, kd, dev, H = _q8_rows(where, q, cache, batch)
    N, D = batch.num_rows, cache.head_dim
    if workspace is None:
        raise ValueError(f"{where}: pass a workspace (see binding.paged_attention_q8_workspace)")
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise TypeError(f"{where}: the workspace must be a contiguous tensor on the tensors' device")
    shape = (N, H, D)
    qs, os_ = q.stride(), out.stride()
    if not (out.dtype is dt and q.get_device() == out.get_device() == dev and
            q.shape == shape == out.shape and qs[2] == os_[2] == 1 and
            (qs[1] == os_[1] == D or H == 1)):
        _bad_rows(where, dt, dev, q=(q, shape), out=(out, shape))
    if N > 1:
        qs, os_ = qs[0], os_[0]
    else:  # (the stride of a single row says nothing)
        qs = os_ = H * D
    qp, op = q.data_ptr(), out.data_ptr()
    if qp == op and N > 0:
        raise ValueError(f"{where}: out must not overlap q")
    rc = cache._call[0](qp, qs, kd, cache._addr, batch._addr, op, os_, H, workspace.data_ptr(),
                        workspace.nbytes, 0 if d_status is None else _status_ptr(d_status),
                        _get_stream(dev) if stream is None else _stream(stream))
    if rc != KVS_OK:
        raise KvsError(rc, where)
    return out


def _vector(t, name, dtype, n, dev):
    """Pointer of a contiguous vector of n entries (n None: any)."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or \
            (n is not None and t.numel() != n):
        raise TypeError(f"{name}: need a contiguous {dtype} vector{'' if n is None else f' of {n}'} "
                        f"on the logits' device, got {tuple(t.shape)} {t.dtype} {t.device}")
    return t.data_ptr()


# kvs_logit_rules: eleven pointers, three 32-bit counts, padding
_pack_rules = struct.Struct("@11Q3i4x").pack


def kvs_process_logits(logits, out=None, token_ids=None, history=None, history_offsets=None,
                       prompt_lens=None, repetition=None, presence=None, frequency=None,
                       bias_ids=None, bias_values=None, bias_offsets=None, mask=None,
                       mask_rows=None, d_status=None, stream=None):
    """Penalties, biases and grammar masks on logits [M, V] (float32, float16 or bfloat16; rows may
    be strided) into out (logits itself is fine; None: only the tokens), and the greedy token of
    the result into token_ids (int32 [M], made when None).  Returns token_ids."""
    dt = _DTYPES.get(logits.dtype)
    if dt is None or not logits.is_cuda or logits.dim() != 2:
        raise TypeError("logits: need a CUDA matrix [M, V] of float32, float16 or bfloat16")
    dev = logits.get_device()
    _call_device(dev, "kvs_process_logits")
    shape = logits.shape
    M, V = shape
    ls = V if logits.is_contiguous() else _row_stride(logits, "logits")
    op = os_ = 0
    if out is not None:
        if out.dtype is not logits.dtype or out.shape != shape or out.get_device() != dev:
            raise TypeError("out: need a matrix like logits")
        op, os_ = out.data_ptr(), V if out.is_contiguous() else _row_stride(out, "out")
    if token_ids is None:
        token_ids = torch.empty(M, dtype=torch.int32, device=logits.device)
    i32, f32 = torch.int32, torch.float32
    h = ho = pl = rp = pr = fr = bi = bv = bo = mp = mr = nh = nb = nm = 0
    if history is not None and history_offsets is not None:
        h, nh = _vector(history, "history", i32, None, dev), history.numel()
        ho = _vector(history_offsets, "history_offsets", i32, M + 1, dev)
    elif history is not None or history_offsets is not None:
        raise ValueError("kvs_process_logits: history and history_offsets come together")
    if prompt_lens is not None:
        pl = _vector(prompt_lens, "prompt_lens", i32, M, dev)
    if repetition is not None:
        rp = _vector(repetition, "repetition", f32, M, dev)
    if presence is not None:
        pr = _vector(presence, "presence", f32, M, dev)
    if frequency is not None:
        fr = _vector(frequency, "frequency", f32, M, dev)
    if bias_ids is not None and bias_values is not None and bias_offsets is not None:
        bi, nb = _vector(bias_ids, "bias_ids", i32, None, dev), bias_ids.numel()
        bv = _vector(bias_values, "bias_values", f32, nb, dev)
        bo = _vector(bias_offsets, "bias_offsets", i32, M + 1, dev)
    elif not (bias_ids is None and bias_values is None and bias_offsets is None):
        raise ValueError("kvs_process_logits: bias_ids, bias_values and bias_offsets come together")
    if mask is not None:
        if mask.dtype is not i32 or mask.get_device() != dev or mask.dim() != 2 or \
                mask.shape[1] != (V + 31) // 32 or not mask.is_contiguous():
            raise TypeError("mask: need a contiguous int32 matrix [masks, ceil(V / 32)] on the "
                            "logits' device")
        mp, nm = mask.data_ptr(), mask.shape[0]
    if mask_rows is not None:
        mr = _vector(mask_rows, "mask_rows", i32, M, dev)
    rules = _pack_rules(h, ho, pl, rp, pr, fr, bi, bv, bo, mp, mr, nh, nb, nm)
    rc = lib().kvs_process_logits(logits.data_ptr(), ls, op, os_, dt, M, V, rules,
                                  _vector(token_ids, "token_ids", i32, M, dev),
                                  0 if d_status is None else _status_ptr(d_status),
                                  _get_stream(dev) if stream is None else _stream(stream))
    if rc != KVS_OK:
        raise KvsError(rc, "kvs_process_logits")
    return token_ids


# kvs_sample_rules: four pointers
_pack_sample = struct.Struct("@4Q").pack


def kvs_sample_logits(logits, uniforms, token_ids=None, temperature=None, top_k=None, top_p=None,
                      min_p=None, token_probs=None, probs=None, stream=None):
    """A token drawn from each row of logits [M, V] (float32, float16 or bfloat16; rows may be
    strided) with the random numbers uniforms (float32 [M], from [0, 1)) into token_ids (int32 [M],
    made when None), under temperature, top_k (int32), top_p and min_p ([M] each, or None).
    token_probs (float32 [M]) gets the tokens' probabilities, probs (float32 [M, V]) those of all
    ids.  Returns token_ids."""
    dt = _DTYPES.get(logits.dtype)
    if dt is None or not logits.is_cuda or logits.dim() != 2:
        raise TypeError("logits: need a CUDA matrix [M, V] of float32, float16 or bfloat16")
    dev = logits.get_device()
    _call_device(dev, "kvs_sample_logits")
    M, V = logits.shape
    ls = V if logits.is_contiguous() else _row_stride(logits, "logits")
    f32, i32 = torch.float32, torch.int32
    pp = ps = 0
    if probs is not None:
        if probs.dtype is not f32 or probs.shape != logits.shape or probs.get_device() != dev:
            raise TypeError("probs: need a float32 matrix [M, V] on the logits' device")
        pp, ps = probs.data_ptr(), V if probs.is_contiguous() else _row_stride(probs, "probs")
    if token_ids is None:
        token_ids = torch.empty(M, dtype=i32, device=logits.device)
    rules = _pack_sample(
        0 if temperature is None else _vector(temperature, "temperature", f32, M, dev),
        0 if top_k is None else _vector(top_k, "top_k", i32, M, dev),
        0 if top_p is None else _vector(top_p, "top_p", f32, M, dev),
        0 if min_p is None else _vector(min_p, "min_p", f32, M, dev))
    lp, ip = logits.data_ptr(), _vector(token_ids, "token_ids", i32, M, dev)
    op = 0 if token_probs is None else _vector(token_probs, "token_probs", f32, M, dev)
    row, step = V * logits.element_size(), ls * logits.element_size()
    for p in (ip, op):  # (the library looks for every other overlap)
        at = p - lp
        if p and -4 * M < at < (M - 1) * step + row and not (row <= at % step <= step - 4 * M):
            raise ValueError("kvs_sample_logits: token_ids and token_probs must not overlap logits")
    rc = lib().kvs_sample_logits(
        lp, ls, dt, M, V, _vector(uniforms, "uniforms", f32, M, dev), rules, ip, op, pp, ps,
        _get_stream(dev) if stream is None else _stream(stream))
    if rc != KVS_OK:
        raise KvsError(rc, "kvs_sample_logits")
    return token_ids


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Row stride of a matrix whose rows are contiguous."""
    s0, s1 = t.stride()
    if s1 != 1 and t.shape[1] > 1:
        raise TypeError(f"{name}: the rows must be contiguous, got strides {t.stride()}")
    return s0 if t.shape[0] > 1 else t.shape[1]
