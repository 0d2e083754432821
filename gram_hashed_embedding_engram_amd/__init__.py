"""Python binding of libengram.so, the gfx950 engram hot path.

Argument marshalling only: torch tensors provide device memory and the
current HIP stream; every step of the path runs in the library's kernels.
The names follow the C ABI in include/engram.h.  There is no fallback: if
the library is not built, every call raises.
"""
import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libengram.so")

OK = 0
E_ARG, E_RANGE, E_UNSUPPORTED, E_STATE, E_HIP, E_DEVICE = -1, -2, -3, -4, -5, -6
DEVERR_TOKEN, DEVERR_ROW, DEVERR_POSITION = 1, 2, 4
DEVERR_PAGE, DEVERR_SEQUENCE = 8, 16
DEVERR_ROUTE = 32
FMT_Q2K, FMT_E4M3 = 0, 1
Q2K_ROW_BYTES = 84
STREAM_ROW_BYTES = 12288      # engram_stream_read's row (ENGRAM_STREAM_ROW_BYTES)
STREAM_SINK_WORDS = 8192      # its sink (ENGRAM_STREAM_SINK_WORDS)
STATIC_SCRATCH_BYTES = 32 << 20   # engram_layer_static's scratch (ENGRAM_STATIC_SCRATCH_BYTES)
PAGE_TOKENS = 64              # positions a cache page holds (ENGRAM_PAGE_TOKENS)
NORM_GROUP = 32               # values a scale of 8- and 4-bit rows covers (ENGRAM_NORM_GROUP)
F8_BLOCK = 128                # weights and values a scale of 8-bit weights covers each way (ENGRAM_F8_BLOCK)
STAGES = ("hash", "gather", "project", "gate")

# Every symbol include/engram.h declares.
EXPORTS = (
    "engram_last_error", "engram_abi_version", "engram_hash", "engram_hash_batch",
    "engram_gather_dequant",
    "engram_project", "engram_project_q2k", "engram_dequant_q2k", "engram_qk_product",
    "engram_gate_apply", "engram_workspace_bytes",
    "engram_ctx_create", "engram_ctx_add_layer", "engram_ctx_set_wkv_q2k", "engram_reset",
    "engram_forward",
    "engram_check", "engram_position", "engram_ctx_buffers", "engram_ctx_set_fused_decode",
    "engram_ctx_set_timing",
    "engram_ctx_timing", "engram_ctx_destroy", "engram_map_host", "engram_stream_read",
    "engram_ctx_set_graph_mode", "engram_ctx_set_position", "engram_layer_static",
    "engram_add_norm", "engram_project_w4", "engram_cache_append", "engram_cache_attend_bytes",
    "engram_cache_attend",
    "engram_project_f8", "engram_route_bytes", "engram_route", "engram_experts_up",
    "engram_experts_down_bytes", "engram_experts_down",
)


class EngramError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"engram error {code}: {msg}")
        self.code = code


class HashTablesC(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("max_ngram", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("vocab", ctypes.c_int64), ("pad_id", ctypes.c_int64),
                ("d_token_map", ctypes.c_void_p), ("multipliers", ctypes.c_void_p),
                ("primes", ctypes.c_void_p), ("offsets", ctypes.c_void_p)]


class TableC(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("scale_block", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("n_rows", ctypes.c_int64), ("d_data", ctypes.c_void_p),
                ("d_scales", ctypes.c_void_p)]


class ConfigC(ctypes.Structure):
    _fields_ = [("hc", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dim", ctypes.c_int64),
                ("eps", ctypes.c_float), ("batch", ctypes.c_int32),
                ("max_tokens", ctypes.c_int64), ("max_seq", ctypes.c_int64),
                ("hash", HashTablesC)]


class CacheC(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_pages", ctypes.c_int64), ("d_k", ctypes.c_void_p), ("d_v", ctypes.c_void_p),
                ("d_k_scales", ctypes.c_void_p), ("d_v_scales", ctypes.c_void_p)]


class SequencesC(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("d_pages", ctypes.c_void_p), ("d_start", ctypes.c_void_p),
                ("d_cu", ctypes.c_void_p), ("d_err", ctypes.c_void_p)]


class RoutesC(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int32), ("chosen", ctypes.c_int32),
                ("tokens", ctypes.c_int64), ("d_ids", ctypes.c_void_p),
                ("d_weights", ctypes.c_void_p), ("d_offsets", ctypes.c_void_p),
                ("d_order", ctypes.c_void_p), ("d_err", ctypes.c_void_p)]


_lib = None
ABI_VERSION = 7           # ENGRAM_ABI_VERSION of include/engram.h this binding follows


def lib():
    """The loaded libengram.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run python -m "
                               "gram_hashed_embedding_engram_amd.build (the engram path has no "
                               "non-HIP fallback)")
        L = ctypes.CDLL(LIB_PATH)
        p, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        sig = {
            "engram_last_error": (ctypes.c_char_p, []),
            "engram_abi_version": (i32, []),
            "engram_hash": (i32, [p, p, i64, i64, p, i64, p, p, p]),
            "engram_hash_batch": (i32, [p, p, i64, i64, i64, p, i64, p, p, p]),
            "engram_gather_dequant": (i32, [p, p, i64, i32, i64, p, p, p]),
            "engram_project": (i32, [p, p, p, i64, i64, i64, p]),
            "engram_project_q2k": (i32, [p, p, p, i64, i64, i64, p]),
            "engram_dequant_q2k": (i32, [p, i64, p, p]),
            "engram_qk_product": (i32, [p, p, p, i64, p]),
            "engram_gate_apply": (i32, [p, p, p, i64, i32, i64, ctypes.c_float, p]),
            "engram_workspace_bytes": (ctypes.c_size_t, [p]),
            "engram_ctx_create": (i32, [p, p, ctypes.c_size_t, p]),
            "engram_ctx_add_layer": (i32, [p, i32, p, p, p]),
            "engram_ctx_set_wkv_q2k": (i32, [p, i32, p]),
            "engram_reset": (i32, [p, p]),
            "engram_forward": (i32, [p, i32, p, i64, p, p]),
            "engram_check": (i32, [p, p]),
            "engram_position": (i64, [p]),
            "engram_ctx_buffers": (i32, [p, p, p, p, p]),
            "engram_ctx_set_fused_decode": (i32, [p, i32]),
            "engram_ctx_set_timing": (i32, [p, i32]),
            "engram_ctx_timing": (i32, [p, p, p]),
            "engram_ctx_destroy": (None, [p]),
            "engram_map_host": (i32, [p, p]),
            "engram_stream_read": (i32, [p, i64, p, p]),
            "engram_ctx_set_graph_mode": (i32, [p, i32, p]),
            "engram_ctx_set_position": (i32, [p, i64, p]),
            "engram_layer_static": (i32, [p, i32, p, p, p, i32, i64, ctypes.c_float, p, i64,
                                          i64, p, i64, p, p, p]),
            "engram_add_norm": (i32, [p, p, i32, p, ctypes.c_float, p, p, p, i64, i64, p]),
            "engram_project_w4": (i32, [p, p, p, p, p, i64, i64, i64, p]),
            "engram_cache_append": (i32, [p, p, p, i64, i64, p, i64, i64, p, i64, i64, p, i32, p,
                                          i32, i32, i64, p]),
            "engram_cache_attend_bytes": (ctypes.c_size_t, [p, p, i32, i64]),
            "engram_cache_attend": (i32, [p, p, p, i64, i64, p, i32, i64, ctypes.c_float, i64, p,
                                          ctypes.c_size_t, p]),
            "engram_project_f8": (i32, [p, p, i32, p, p, p, i64, i64, i64, p]),
            "engram_route_bytes": (ctypes.c_size_t, [p]),
            "engram_route": (i32, [p, p, i32, i64, p, i32, i32, i32, i32, i32, ctypes.c_float, p,
                                   ctypes.c_size_t, p]),
            "engram_experts_up": (i32, [p, p, p, i32, p, p, p, p, i64, i64, p]),
            "engram_experts_down_bytes": (ctypes.c_size_t, [p, i64]),
            "engram_experts_down": (i32, [p, p, p, i32, p, p, p, i64, i64, p, ctypes.c_size_t, p]),
        }
        # a library built before this binding: another version, or, as additions
        # alone leave the version as it is, one that lacks an entry point
        rebuild = "rebuild it (python -m gram_hashed_embedding_engram_amd.build)"
        if L.engram_abi_version() != ABI_VERSION:
            raise RuntimeError(f"{LIB_PATH} has ABI version {L.engram_abi_version()}, this "
                               f"binding {ABI_VERSION}: {rebuild}")
        for name, (res, args) in sig.items():
            if not hasattr(L, name):
                raise RuntimeError(f"{LIB_PATH} has no {name}: {rebuild}")
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def last_error() -> str:
    return lib().engram_last_error().decode()


def _check(rc):
    if rc != OK:
        raise EngramError(rc, last_error())


def _ptr(t):
    """Device (or host numpy) address of a tensor / array; None -> NULL."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _room(t):
    """Bytes from a tensor's (or array's) first element to the end of its
    storage: what a kernel may touch through its address."""
    if isinstance(t, np.ndarray):
        return t.nbytes if t.flags.c_contiguous else -1
    return t.untyped_storage().nbytes() - t.storage_offset() * t.element_size()


def _need(t, name, nbytes, dense=True):
    """Refuse, before the library sees the address, a tensor that a call of
    these sizes would read or write past the end of its storage, or a strided
    view where the kernel takes rows to be back to back.  The C entry points
    cannot see a buffer's size; the binding can."""
    if t is None:
        return
    if dense and not isinstance(t, np.ndarray) and not t.is_contiguous():
        raise EngramError(E_ARG, f"{name}: a contiguous tensor is needed")
    room = _room(t)
    if nbytes > room:
        raise EngramError(E_ARG, f"{name}: the call needs {nbytes} bytes, its storage holds "
                                 f"{max(room, 0)} from this address")


_current = None


def _stream(stream):
    global _current
    if stream is None:
        if _current is None:
            import torch
            first = torch.cuda.current_stream().cuda_stream      # initialises the device
            # the same address without a Stream object a call (0.2 us, not 3), where
            # torch has these two functions of its own
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            device = getattr(torch._C, "_cuda_getDevice", None)
            if raw and device:
                _current = lambda: raw(device())  # noqa: E731
            else:
                _current = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
            return first
        return _current()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class HashTables:
    """Hash tables for the ABI: token_map on the device (torch int64
    tensor), multipliers / primes / offsets as host arrays."""

    def __init__(self, d_token_map, pad_id, multipliers, primes, offsets):
        self.mult = np.ascontiguousarray(multipliers, dtype=np.int64)
        self.primes = np.ascontiguousarray(primes, dtype=np.int64)
        self.offsets = np.ascontiguousarray(offsets, dtype=np.int64)
        self.token_map = d_token_map
        self.n_layers, self.max_ngram = self.mult.shape
        self.cols = self.primes.shape[1]
        self.n_heads = self.cols // (self.max_ngram - 1)
        self.c = HashTablesC(self.n_layers, self.max_ngram, self.n_heads, 0,
                             int(d_token_map.numel()), int(pad_id), _ptr(d_token_map),
                             self.mult.ctypes.data, self.primes.ctypes.data,
                             self.offsets.ctypes.data)


def map_host(t):
    """Device address of a pinned host tensor (engram_map_host)."""
    dev = ctypes.c_void_p()
    _check(lib().engram_map_host(ctypes.c_void_p(t.data_ptr()), ctypes.byref(dev)))
    return dev.value


def _table_ptr(t):
    if t is None:
        return None
    return t.data_ptr() if t.is_cuda else map_host(t)


class Table:
    """One layer's table (Q2_K blocks, or e4m3 codes with f32 block scales),
    as device tensors or as pinned host tensors the kernels read across the
    host link."""

    def __init__(self, d_data, d_scales=None, head_dim=256, scale_block=128):
        fmt = FMT_Q2K if d_scales is None else FMT_E4M3
        n_rows = int(d_data.shape[0])
        self.data, self.scales = d_data, d_scales
        self.c = TableC(fmt, head_dim, scale_block if fmt == FMT_E4M3 else 0, 0, n_rows,
                        _table_ptr(d_data), _table_ptr(d_scales))


def hash(tables: HashTables, d_ids, start_pos, d_history, d_row_ids, d_err=None, stream=None):
    T = int(d_ids.numel())
    _need(d_ids, "ids", 4 * T)
    _need(d_history, "history", 8 * int(d_history.numel()))
    _need(d_row_ids, "row_ids", 8 * T * tables.n_layers * tables.cols)
    _need(d_err, "err", 4)
    _check(lib().engram_hash(ctypes.byref(tables.c), _ptr(d_ids), int(d_ids.numel()),
                             int(start_pos), _ptr(d_history), int(d_history.numel()),
                             _ptr(d_row_ids), _ptr(d_err), _stream(stream)))


def hash_batch(tables: HashTables, d_ids, start_pos, d_history, d_row_ids, d_err=None,
               stream=None):
    """d_ids [B, T] int32, d_history [B, max_seq] int64, d_row_ids [B*T, nl, cols]."""
    B, T = d_ids.shape
    _need(d_ids, "ids", 4 * B * T)
    _need(d_history, "history", 8 * B * d_history.shape[1])
    _need(d_row_ids, "row_ids", 8 * B * T * tables.n_layers * tables.cols)
    _need(d_err, "err", 4)
    _check(lib().engram_hash_batch(ctypes.byref(tables.c), _ptr(d_ids), int(B), int(T),
                                   int(start_pos), _ptr(d_history), int(d_history.shape[1]),
                                   _ptr(d_row_ids), _ptr(d_err), _stream(stream)))


def gather_dequant(table: Table, d_row_ids, T, cols, id_stride, d_rows, d_err=None,
                   stream=None):
    if T > 0:
        # ids of token t at d_row_ids + t*id_stride: any view that reaches them will do
        _need(d_row_ids, "row_ids", 8 * ((T - 1) * id_stride + cols), dense=False)
        _need(d_rows, "rows", 2 * T * cols * table.c.head_dim)
    _need(d_err, "err", 4)
    _check(lib().engram_gather_dequant(ctypes.byref(table.c), _ptr(d_row_ids), int(T),
                                       int(cols), int(id_stride), _ptr(d_rows), _ptr(d_err),
                                       _stream(stream)))


def project(d_x, d_w, d_y, stream=None):
    T, K = d_x.shape
    N = d_w.shape[0]
    _need(d_x, "x", 2 * T * K)
    _need(d_w, "w", 2 * N * K)
    _need(d_y, "y", 2 * T * N)
    _check(lib().engram_project(_ptr(d_x), _ptr(d_w), _ptr(d_y), T, K, N, _stream(stream)))


def project_q2k(d_x, d_wq, d_y, stream=None):
    """d_x [T, K] bf16 bits (T <= 1), d_wq [N, K/256, 84] uint8 Q2_K blocks."""
    T, K = d_x.shape
    N = d_wq.shape[0]
    _need(d_x, "x", 2 * T * K)
    _need(d_wq, "wkv_q2k", N * (K // 256) * 84)
    _need(d_y, "y", 2 * T * N)
    _check(lib().engram_project_q2k(_ptr(d_x), _ptr(d_wq), _ptr(d_y), T, K, N, _stream(stream)))


def dequant_q2k(d_blocks, d_out, stream=None):
    """Q2_K blocks (any shape [..., 84] uint8) -> d_out [n_blocks * 256] bf16 bits."""
    n = d_blocks.numel() // 84
    _need(d_blocks, "blocks", 84 * n)
    _need(d_out, "out", 2 * 256 * n)
    _check(lib().engram_dequant_q2k(_ptr(d_blocks), n, _ptr(d_out), _stream(stream)))


def qk_product(d_q, d_k, d_qk, stream=None):
    n = int(d_q.numel())
    _need(d_q, "q", 2 * n)
    _need(d_k, "k", 2 * n)
    _need(d_qk, "qk", 4 * n)
    _check(lib().engram_qk_product(_ptr(d_q), _ptr(d_k), _ptr(d_qk), int(d_q.numel()),
                                   _stream(stream)))


def stream_read(d_src, d_sink, stream=None):
    """Stream d_src once, one XOR fold per wavefront into d_sink [8192]
    int32 (the read-rate yardstick; engram_stream_read)."""
    _need(d_sink, "sink", 4 * STREAM_SINK_WORDS)
    _check(lib().engram_stream_read(_ptr(d_src), int(d_src.numel() * d_src.element_size()),
                                    _ptr(d_sink), _stream(stream)))


def gate_apply(d_h, d_kv, d_qk, eps, stream=None):
    T, hc, dim = d_h.shape
    _need(d_h, "h", 4 * T * hc * dim)
    _need(d_kv, "kv", 2 * T * dim * (hc + 1))
    _need(d_qk, "qk", 4 * hc * dim)
    _check(lib().engram_gate_apply(_ptr(d_h), _ptr(d_kv), _ptr(d_qk), T, hc, dim,
                                   float(eps), _stream(stream)))


def layer_static(tables: HashTables, hash_index, table: Table, d_wkv, d_qk, eps, d_ids,
                 start_pos, d_history, d_h, d_err=None, stream=None):
    """One engram layer over d_ids [T] at start_pos with its row ids, rows
    and kv in the library's static scratch (engram_layer_static: allocates
    nothing).  d_history [max_seq] int64, d_h [T, hc, dim] f32 in place."""
    T = int(d_ids.numel())
    _, hc, dim = d_h.shape
    K = tables.cols * table.c.head_dim
    _need(d_ids, "ids", 4 * T)
    _need(d_history, "history", 8 * int(d_history.numel()))
    _need(d_wkv, "wkv", 2 * dim * (hc + 1) * K)
    _need(d_qk, "qk", 4 * hc * dim)
    _need(d_h, "h", 4 * T * hc * dim)
    _need(d_err, "err", 4)
    _check(lib().engram_layer_static(ctypes.byref(tables.c), int(hash_index),
                                     ctypes.byref(table.c), _ptr(d_wkv), _ptr(d_qk), int(hc),
                                     int(dim), float(eps), _ptr(d_ids), T, int(start_pos),
                                     _ptr(d_history), int(d_history.numel()), _ptr(d_h),
                                     _ptr(d_err), _stream(stream)))


# The attention sub-layer's calls look at all their tensors in one condition and
# go through _typed and _heads, one by one, only to name what is wrong: a call of
# a function a tensor would cost as much as the launch.
def _typed(t, name, dtypes, shape=None):
    """Refuse a tensor of another type, shape or, for the kernels that take
    rows back to back, a strided view."""
    if t.dtype not in dtypes:
        kinds = ", ".join(sorted(str(d)[6:] for d in dtypes))
        raise EngramError(E_ARG, f"{name}: {t.dtype}, one of {kinds} is needed")
    if shape is not None and t.shape != shape:
        raise EngramError(E_ARG, f"{name}: shape {tuple(t.shape)}, {tuple(shape)} is needed")
    if not t.is_contiguous():
        raise EngramError(E_ARG, f"{name}: a contiguous tensor is needed")


def _on_gpu(t, name):
    """Refuse a tensor in host memory, whose address a kernel cannot read."""
    if not t.is_cuda:
        raise EngramError(E_ARG, f"{name}: a tensor on the GPU is needed, this one is on {t.device}")


def _host_name(**tensors):
    """The name of the first of these tensors that is in host memory, or None:
    what W4, Cache and Sequences keep, so that a call need not look again."""
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            return name.replace("_", " ")
    return None


def _refuse_host(*names):
    for name in names:
        if name is not None:
            raise EngramError(E_ARG, f"{name}: a tensor on the GPU is needed, this one is not")


class _Types:
    """Element types the attention sub-layer's tensors may have (torch is
    imported by the first call that needs it)."""

    def __init__(self):
        import torch as t
        self.f32 = frozenset((t.float32,))
        self.i32 = frozenset((t.int32,))
        self.u8 = frozenset((t.uint8,))
        self.bf16 = frozenset((t.bfloat16, t.int16))       # bf16 values or their bits
        self.res = self.f32 | self.bf16
        self.e4m3 = frozenset((t.uint8, t.float8_e4m3fn))
        self.e8m0 = frozenset((t.uint8, t.float8_e8m0fnu))


_types = None


def _kinds():
    global _types
    if _types is None:
        _types = _Types()
    return _types


def add_norm(d_x, d_res, d_w, eps, d_codes, d_scales, d_sum=None, stream=None):
    """Residual addition, root-mean-square norm and 8-bit output
    (engram_add_norm): d_sum = d_res + d_x, d_codes / d_scales = the normed
    sum in e4m3 with a scale per 32 values.  d_res [..., dim] f32 or bf16,
    d_x bf16 of the same shape or None, d_sum None = in place on d_res."""
    k = _types or _kinds()
    shape = d_res.shape
    dim = shape[-1]
    groups = shape[:-1] + (dim // NORM_GROUP,)
    total = d_res if d_sum is None else d_sum
    if not (d_res.dtype in k.res and d_res.is_cuda and d_res.is_contiguous()
            and (total is d_res or total.dtype is d_res.dtype and total.is_cuda
                 and total.shape == shape and total.is_contiguous())
            and (d_x is None or d_x.dtype in k.bf16 and d_x.is_cuda and d_x.shape == shape
                 and d_x.is_contiguous())
            and d_w.dtype in k.bf16 and d_w.is_cuda and d_w.shape == (dim,) and d_w.is_contiguous()
            and d_codes.dtype in k.e4m3 and d_codes.is_cuda and d_codes.shape == shape
            and d_codes.is_contiguous()
            and d_scales.dtype in k.e8m0 and d_scales.is_cuda and d_scales.shape == groups
            and d_scales.is_contiguous()):
        _typed(d_res, "res", k.res)
        _typed(total, "sum", (d_res.dtype,), shape)
        if d_x is not None:
            _typed(d_x, "x", k.bf16, shape)
        _typed(d_w, "w", k.bf16, (dim,))
        _typed(d_codes, "codes", k.e4m3, shape)
        _typed(d_scales, "scales", k.e8m0, groups)
        for t, name in ((d_res, "res"), (total, "sum"), (d_x, "x"), (d_w, "w"), (d_codes, "codes"),
                        (d_scales, "scales")):
            if t is not None:
                _on_gpu(t, name)
    rc = (_lib or lib()).engram_add_norm(
        None if d_x is None else d_x.data_ptr(), d_res.data_ptr(), d_res.dtype not in k.f32,
        d_w.data_ptr(), eps, total.data_ptr(), d_codes.data_ptr(), d_scales.data_ptr(),
        d_res.numel() // dim if dim else 0, dim, _stream(stream))
    if rc:
        _check(rc)


class W4:
    """A weight matrix in 4 bits: d_w [N, K/2] e2m1 codes (the even value in
    the low nibble), d_scales [N, K/32] exponents + 127."""

    def __init__(self, d_w, d_scales):
        N, half = d_w.shape
        k = _kinds()
        _typed(d_w, "w", k.u8)
        _typed(d_scales, "w scales", k.e8m0, (N, 2 * half // NORM_GROUP))
        self.w, self.scales = d_w, d_scales
        self.N, self.K, self.groups = N, 2 * half, 2 * half // NORM_GROUP
        self.at = (d_w.data_ptr(), d_scales.data_ptr())
        self.host = _host_name(w=d_w, w_scales=d_scales)


def project_w4(d_x, weights: W4, d_y, d_xs=None, stream=None):
    """y = x w^T through 4-bit weights (engram_project_w4): d_x [T, K] bf16,
    or e4m3 codes with d_xs [T, K/32]; d_y [T, N] bf16."""
    k = _types or _kinds()
    T, K, N = d_x.shape[0], weights.K, weights.N
    if not ((d_x.dtype in k.bf16 if d_xs is None else
             d_x.dtype in k.e4m3 and d_xs.dtype in k.e8m0 and d_xs.is_cuda
             and d_xs.shape == (T, weights.groups) and d_xs.is_contiguous())
            and d_x.is_cuda and d_x.shape == (T, K) and d_x.is_contiguous()
            and d_y.dtype in k.bf16 and d_y.is_cuda and d_y.shape == (T, N) and d_y.is_contiguous()
            and weights.host is None):
        _typed(d_x, "x", k.bf16 if d_xs is None else k.e4m3, (T, K))
        if d_xs is not None:
            _typed(d_xs, "x scales", k.e8m0, (T, weights.groups))
        _typed(d_y, "y", k.bf16, (T, N))
        _refuse_host(weights.host)
        for t, name in ((d_x, "x"), (d_xs, "x scales"), (d_y, "y")):
            if t is not None:
                _on_gpu(t, name)
    xs = None if d_xs is None else d_xs.data_ptr()
    w, ws = weights.at
    rc = (_lib or lib()).engram_project_w4(d_x.data_ptr(), xs, w, ws, d_y.data_ptr(), T, K, N,
                                           _stream(stream))
    if rc:
        _check(rc)


class Cache:
    """A paged 8-bit cache of keys and values (engram_cache): codes
    [n_pages, kv_heads, 64, head_dim], scales [n_pages, kv_heads] f32."""

    def __init__(self, d_k, d_v, d_k_scales, d_v_scales):
        n_pages, kv_heads, page, head_dim = d_k.shape
        k = _kinds()
        _typed(d_k, "k", k.e4m3, (n_pages, kv_heads, PAGE_TOKENS, head_dim))
        _typed(d_v, "v", k.e4m3, d_k.shape)
        _typed(d_k_scales, "k scales", k.f32, (n_pages, kv_heads))
        _typed(d_v_scales, "v scales", k.f32, (n_pages, kv_heads))
        self.keep = (d_k, d_v, d_k_scales, d_v_scales)
        self.host = _host_name(k=d_k, v=d_v, k_scales=d_k_scales, v_scales=d_v_scales)
        self.kv_heads, self.head_dim, self.n_pages = kv_heads, head_dim, n_pages
        self.c = CacheC(kv_heads, head_dim, n_pages, d_k.data_ptr(), d_v.data_ptr(),
                        d_k_scales.data_ptr(), d_v_scales.data_ptr())
        self.ref = ctypes.byref(self.c)


class Sequences:
    """The sequences of a step (engram_seqs): d_pages [B, max_pages] int32,
    d_start [B] int32, d_cu [B+1] int32 token bounds (None: every sequence
    brings as many tokens), d_err an int32 error word or None."""

    def __init__(self, d_pages, d_start, d_cu=None, d_err=None):
        B, width = d_pages.shape
        i32 = _kinds().i32
        _typed(d_pages, "pages", i32)
        _typed(d_start, "start", i32, (B,))
        if d_cu is not None:
            _typed(d_cu, "cu", i32, (B + 1,))
        if d_err is not None:
            _typed(d_err, "err", i32)
            _need(d_err, "err", 4)
        self.keep = (d_pages, d_start, d_cu, d_err)
        self.host = _host_name(pages=d_pages, start=d_start, cu=d_cu, err=d_err)
        self.B = B
        self.c = SequencesC(B, width, d_pages.data_ptr(), d_start.data_ptr(), _ptr(d_cu),
                            _ptr(d_err))
        self.ref = ctypes.byref(self.c)


def _heads(t, name, T, heads, head_dim):
    """(address, token stride, head stride) of bf16 heads [T, heads, head_dim]
    that may be a view of a wider row; a head's values lie side by side."""
    if t.dtype not in _types.bf16:
        raise EngramError(E_ARG, f"{name}: {t.dtype}, bfloat16 is needed")
    if t.shape != (T, heads, head_dim):
        raise EngramError(E_ARG, f"{name}: shape {tuple(t.shape)}, {(T, heads, head_dim)} is needed")
    token, head, one = t.stride()
    if one != 1:
        raise EngramError(E_ARG, f"{name}: a head's values must lie side by side")
    if not t.is_cuda:
        _on_gpu(t, name)
    return t.data_ptr(), token, head


def cache_append(cache: Cache, seqs: Sequences, d_k, d_v, d_freq, d_q=None, d_q_out=None,
                 halves=True, stream=None):
    """Rotates the step's queries and keys and appends its keys and values to
    the cache (engram_cache_append).  d_k, d_v [T, kv_heads, head_dim] and d_q
    [T, q_heads, head_dim] bf16, as views of one projection's output if need
    be; d_freq [rot/2] f32 or None (no rotation); d_q_out as d_q, contiguous."""
    T, kv, d = d_k.shape[0], cache.kv_heads, cache.head_dim
    if cache.host is not None or seqs.host is not None:
        _refuse_host(cache.host, seqs.host)
    kp, kt, kh = _heads(d_k, "k", T, kv, d)
    vp, vt, vh = _heads(d_v, "v", T, kv, d)
    qp = qt = qh = q_heads = qo = 0
    if d_q is not None:
        q_heads = d_q.shape[1]
        qp, qt, qh = _heads(d_q, "q", T, q_heads, d)
        if d_q_out is None:
            raise EngramError(E_ARG, "q_out: queries are given and no place for them")
        _typed(d_q_out, "q_out", _types.bf16, (T, q_heads, d))
        _on_gpu(d_q_out, "q_out")
        qo = d_q_out.data_ptr()
    rot = fp = 0
    if d_freq is not None:
        _typed(d_freq, "freq", _types.f32)
        _on_gpu(d_freq, "freq")
        rot, fp = 2 * d_freq.numel(), d_freq.data_ptr()
    rc = (_lib or lib()).engram_cache_append(cache.ref, seqs.ref, kp, kt, kh, vp, vt, vh, qp, qt, qh, qo,
                                  q_heads, fp, rot, halves, T, _stream(stream))
    if rc:
        _check(rc)


def cache_attend_bytes(cache: Cache, seqs: Sequences, q_heads, T):
    """Workspace bytes a cache_attend of T tokens needs (may be 0)."""
    return lib().engram_cache_attend_bytes(cache.ref, seqs.ref, int(q_heads), int(T))


def cache_attend(cache: Cache, seqs: Sequences, d_q, d_out, scale, window=0, d_ws=None,
                 stream=None):
    """Attention of the step's queries over the cache (engram_cache_attend):
    d_q [T, q_heads, head_dim] bf16 (a view if need be), d_out contiguous of
    that shape, d_ws a uint8 tensor of cache_attend_bytes bytes or None."""
    T, q_heads, _ = shape = d_q.shape
    if cache.host is not None or seqs.host is not None:
        _refuse_host(cache.host, seqs.host)
    qp, qt, qh = _heads(d_q, "q", T, q_heads, cache.head_dim)
    _typed(d_out, "out", _types.bf16, shape)
    _on_gpu(d_out, "out")
    ws, nws = 0, 0
    if d_ws is not None:
        _typed(d_ws, "ws", _types.u8)
        _on_gpu(d_ws, "ws")
        ws, nws = d_ws.data_ptr(), d_ws.numel()
    rc = (_lib or lib()).engram_cache_attend(cache.ref, seqs.ref, qp, qt, qh, d_out.data_ptr(), q_heads, T,
                                  scale, window, ws, nws, _stream(stream))
    if rc:
        _check(rc)


# The experts' sub-layer's calls, as the attention sub-layer's, look at all their
# tensors in one condition.
class F8:
    """Weight matrices in 8 bits: d_w [..., N, K] e4m3 codes, d_scales
    [..., ceil(N/128), K/128] f32, one per block of 128 x 128."""

    def __init__(self, d_w, d_scales):
        *lead, N, K = d_w.shape
        k = _kinds()
        _typed(d_w, "w", k.e4m3)
        _typed(d_scales, "w scales", k.f32, (*lead, -(-N // F8_BLOCK), -(-K // F8_BLOCK)))
        self.w, self.scales, self.lead = d_w, d_scales, tuple(lead)
        self.N, self.K = N, K
        self.scale_shapes = (K // NORM_GROUP, K // F8_BLOCK)
        self.at = (d_w.data_ptr(), d_scales.data_ptr())
        self.host = _host_name(w=d_w, w_scales=d_scales)
        self.device = _one_device(w=d_w, w_scales=d_scales)


class Routes:
    """Where a step's tokens go (engram_routes): d_ids [T, k] int32 and
    d_weights [T, k] f32, the experts of each token; d_offsets [experts+1] and
    d_order [T*k] int32, their slots sorted by expert; d_err an int32 error
    word or None.  route fills the first four."""

    def __init__(self, d_ids, d_weights, d_offsets, d_order, d_err=None):
        T, chosen = d_ids.shape
        k = _kinds()
        _typed(d_ids, "ids", k.i32)
        _typed(d_weights, "weights", k.f32, (T, chosen))
        _typed(d_offsets, "offsets", k.i32)
        _typed(d_order, "order", k.i32, (T * chosen,))
        if d_offsets.dim() != 1 or d_offsets.numel() < 2:
            raise EngramError(E_ARG, f"offsets: shape {tuple(d_offsets.shape)}, (experts + 1,) is needed")
        if d_err is not None:
            _typed(d_err, "err", k.i32)
            _need(d_err, "err", 4)
        self.keep = (d_ids, d_weights, d_offsets, d_order, d_err)
        self.host = _host_name(ids=d_ids, weights=d_weights, offsets=d_offsets, order=d_order,
                               err=d_err)
        self.device = _one_device(ids=d_ids, weights=d_weights, offsets=d_offsets, order=d_order,
                                  err=d_err)
        self.T, self.k, self.experts = T, chosen, d_offsets.numel() - 1
        self.c = RoutesC(self.experts, chosen, T, d_ids.data_ptr(), d_weights.data_ptr(),
                         d_offsets.data_ptr(), d_order.data_ptr(), _ptr(d_err))
        self.ref = ctypes.byref(self.c)


def _one_device(**tensors):
    """The index of the device that these tensors share (-1: host memory)."""
    first = None
    for name, t in tensors.items():
        if t is not None:
            if first is None:
                first = t.get_device()
            elif t.get_device() != first:
                raise EngramError(E_ARG, f"{name.replace('_', ' ')}: on {t.device}, the others are not")
    return first


_device = None


def _here(device):
    """Refuse a call whose tensors are on another device than the current one,
    whose stream it would be enqueued on."""
    global _device
    if _device is None:
        import torch
        torch.cuda.current_stream()                          # initialises the device
        _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if device != _device():
        raise EngramError(E_ARG, f"the tensors are on device {device}, the current one is {_device()}")


def _rows8(k, x, xs, rows, weights):
    """Whether x and xs are such rows: 0 with E8M0 scales, 1 with f32 ones, -1 neither."""
    if not (x.dtype in k.e4m3 and x.shape == (rows, weights.K) and x.is_contiguous()
            and xs.is_contiguous()):
        return -1
    if xs.dtype in k.f32:
        return 1 if xs.shape == (rows, weights.scale_shapes[1]) else -1
    return 0 if xs.dtype in k.e8m0 and xs.shape == (rows, weights.scale_shapes[0]) else -1


def _refuse_rows8(k, x, xs, name, rows, weights):
    _typed(x, name, k.e4m3, (rows, weights.K))
    _typed(xs, name + " scales", k.e8m0 | k.f32,
           (rows, weights.scale_shapes[xs.dtype in k.f32]))


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None:
            _on_gpu(t, name.replace("_", " "))
            if t.get_device() != device:
                raise EngramError(E_ARG, f"{name.replace('_', ' ')}: on {t.device}, not on the "
                                         f"call's device {device}")


def project_f8(d_x, weights: F8, d_y, d_xs, stream=None):
    """y = x w^T through 8-bit weights (engram_project_f8): d_x [T, K] e4m3
    codes with d_xs [T, K/32] (powers of two, as add_norm gives them) or
    [T, K/128] f32; d_y [T, N] bf16."""
    k = _types or _kinds()
    T, dev = d_x.shape[0], weights.device
    kind = _rows8(k, d_x, d_xs, T, weights)
    if not (kind >= 0 and dev >= 0 and weights.lead == () and weights.host is None
            and d_y.dtype in k.bf16 and d_y.shape == (T, weights.N) and d_y.is_contiguous()
            and d_x.get_device() == dev and d_xs.get_device() == dev and d_y.get_device() == dev):
        if weights.lead:
            raise EngramError(E_ARG, f"w: {weights.lead} matrices, one is needed")
        _refuse_rows8(k, d_x, d_xs, "x", T, weights)
        _typed(d_y, "y", k.bf16, (T, weights.N))
        _refuse_host(weights.host)
        _same_device(dev, x=d_x, x_scales=d_xs, y=d_y)
    _here(dev)
    w, ws = weights.at
    rc = (_lib or lib()).engram_project_f8(d_x.data_ptr(), d_xs.data_ptr(), kind, w, ws,
                                           d_y.data_ptr(), T, weights.K, weights.N,
                                           _stream(stream))
    if rc:
        _check(rc)


def route_bytes(routes: Routes):
    """Workspace bytes a route of these sizes needs (may be 0)."""
    return lib().engram_route_bytes(routes.ref)


def route(d_logits, routes: Routes, d_bias=None, softmax=False, groups=1, top_groups=1,
          group_best=2, renorm=True, factor=1.0, d_ws=None, stream=None):
    """Routing to experts (engram_route): d_logits [T, experts] f32 or bf16 (a
    view of wider rows if need be), d_bias [experts] f32 or None; fills
    routes.  Scores are sigmoids, or with softmax=True softmaxes; of `groups`
    runs of experts the top_groups with the largest sum of their group_best
    best are kept.  d_ws a uint8 tensor of route_bytes bytes or None."""
    k = _types or _kinds()
    dev = routes.device
    if not (d_logits.dtype in k.res and d_logits.shape == (routes.T, routes.experts)
            and routes.host is None and dev >= 0 and d_logits.get_device() == dev
            and (d_logits.stride(1) == 1 or routes.experts == 1)
            and (d_bias is None or d_bias.dtype in k.f32 and d_bias.shape == (routes.experts,)
                 and d_bias.is_contiguous() and d_bias.get_device() == dev)
            and (d_ws is None or d_ws.dtype in k.u8 and d_ws.is_contiguous()
                 and d_ws.get_device() == dev)):
        if d_logits.dtype not in k.res:
            _typed(d_logits, "logits", k.res)
        if d_logits.shape != (routes.T, routes.experts):
            raise EngramError(E_ARG, f"logits: shape {tuple(d_logits.shape)}, "
                                     f"{(routes.T, routes.experts)} is needed")
        if routes.experts > 1 and d_logits.stride(1) != 1:
            raise EngramError(E_ARG, "logits: a row's values must lie side by side")
        if d_bias is not None:
            _typed(d_bias, "bias", k.f32, (routes.experts,))
        if d_ws is not None:
            _typed(d_ws, "ws", k.u8)
        _refuse_host(routes.host)
        _same_device(dev, logits=d_logits, bias=d_bias, ws=d_ws)
    _here(dev)
    stride = d_logits.stride(0) if routes.T > 1 else routes.experts
    ws, nws = (0, 0) if d_ws is None else (d_ws.data_ptr(), d_ws.numel())
    rc = (_lib or lib()).engram_route(
        routes.ref, d_logits.data_ptr(), d_logits.dtype not in k.f32, stride,
        None if d_bias is None else d_bias.data_ptr(), softmax, groups, top_groups, group_best,
        renorm, factor, ws, nws, _stream(stream))
    if rc:
        _check(rc)


def experts_up(d_x, d_xs, weights: F8, routes: Routes, d_h, d_hs, stream=None):
    """The experts' gated up projection (engram_experts_up): d_x [T, K] e4m3
    codes with scales d_xs as for project_f8; weights [experts, 2, I, K], the
    gate's and the up matrix; d_h [T*k, I] codes and d_hs [T*k, I/32] in the
    plan's order."""
    k = _types or _kinds()
    T, R, I, dev = routes.T, routes.T * routes.k, weights.N, weights.device
    kind = _rows8(k, d_x, d_xs, T, weights)
    if not (kind >= 0 and dev >= 0 and weights.lead == (routes.experts, 2) and weights.host is None
            and routes.host is None and routes.device == dev
            and d_h.dtype in k.e4m3 and d_h.shape == (R, I) and d_h.is_contiguous()
            and d_hs.dtype in k.e8m0 and d_hs.shape == (R, I // NORM_GROUP) and d_hs.is_contiguous()
            and d_x.get_device() == dev and d_xs.get_device() == dev
            and d_h.get_device() == dev and d_hs.get_device() == dev):
        if weights.lead != (routes.experts, 2):
            raise EngramError(E_ARG, f"w: {weights.lead} matrices, {(routes.experts, 2)} are needed")
        _refuse_rows8(k, d_x, d_xs, "x", T, weights)
        _typed(d_h, "h", k.e4m3, (R, I))
        _typed(d_hs, "h scales", k.e8m0, (R, I // NORM_GROUP))
        _refuse_host(weights.host, routes.host)
        _same_device(dev, x=d_x, x_scales=d_xs, h=d_h, h_scales=d_hs, ids=routes.keep[0])
    _here(dev)
    w, ws = weights.at
    rc = (_lib or lib()).engram_experts_up(routes.ref, d_x.data_ptr(), d_xs.data_ptr(), kind, w, ws,
                                           d_h.data_ptr(), d_hs.data_ptr(), weights.K, I,
                                           _stream(stream))
    if rc:
        _check(rc)


def experts_down_bytes(weights: F8, routes: Routes):
    """Workspace bytes an experts_down of these sizes needs (may be 0)."""
    return lib().engram_experts_down_bytes(routes.ref, weights.N)


def experts_down(d_h, d_hs, weights: F8, routes: Routes, d_y, d_ws=None, stream=None):
    """The experts' down projection and the weighted sum over a token's experts
    (engram_experts_down): d_h [T*k, K] in the plan's order with scales d_hs as
    for project_f8; weights [experts, N, K]; d_y [T, N] bf16; d_ws a uint8
    tensor of experts_down_bytes bytes or None."""
    k = _types or _kinds()
    T, dev = routes.T, weights.device
    kind = _rows8(k, d_h, d_hs, T * routes.k, weights)
    if not (kind >= 0 and dev >= 0 and weights.lead == (routes.experts,) and weights.host is None
            and routes.host is None and routes.device == dev
            and d_y.dtype in k.bf16 and d_y.shape == (T, weights.N) and d_y.is_contiguous()
            and d_h.get_device() == dev and d_hs.get_device() == dev and d_y.get_device() == dev
            and (d_ws is None or d_ws.dtype in k.u8 and d_ws.is_contiguous()
                 and d_ws.get_device() == dev)):
        if weights.lead != (routes.experts,):
            raise EngramError(E_ARG, f"w: {weights.lead} matrices, {(routes.experts,)} are needed")
        _refuse_rows8(k, d_h, d_hs, "h", T * routes.k, weights)
        _typed(d_y, "y", k.bf16, (T, weights.N))
        if d_ws is not None:
            _typed(d_ws, "ws", k.u8)
        _refuse_host(weights.host, routes.host)
        _same_device(dev, h=d_h, h_scales=d_hs, y=d_y, ws=d_ws, ids=routes.keep[0])
    _here(dev)
    w, ws = weights.at
    space, nws = (0, 0) if d_ws is None else (d_ws.data_ptr(), d_ws.numel())
    rc = (_lib or lib()).engram_experts_down(routes.ref, d_h.data_ptr(), d_hs.data_ptr(), kind, w,
                                             ws, d_y.data_ptr(), weights.K, weights.N, space, nws,
                                             _stream(stream))
    if rc:
        _check(rc)


class Context:
    """The stateful engram of one sequence (engram_ctx)."""

    def __init__(self, tables: HashTables, hc, dim, head_dim, eps, max_tokens, max_seq,
                 d_workspace=None, batch=1):
        import torch
        self.tables = tables
        self.batch = batch
        self.cfg = ConfigC(hc, head_dim, dim, eps, batch, max_tokens, max_seq, tables.c)
        nbytes = lib().engram_workspace_bytes(ctypes.byref(self.cfg))
        if nbytes == 0:
            raise EngramError(E_ARG, "invalid engram configuration")
        if d_workspace is None:
            d_workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.workspace = d_workspace
        self.nl, self.cols = tables.n_layers, tables.cols
        self.hc, self.dim, self.head_dim = hc, dim, head_dim
        h = ctypes.c_void_p()
        _check(lib().engram_ctx_create(ctypes.byref(self.cfg), _ptr(d_workspace),
                                       int(d_workspace.numel()), ctypes.byref(h)))
        self.h = h
        self._keep = {}

    def add_layer(self, hash_index, table: Table, d_wkv, d_qk):
        K = self.cols * self.head_dim
        _need(d_wkv, "wkv", 2 * self.dim * (self.hc + 1) * K)
        _need(d_qk, "qk", 4 * self.hc * self.dim)
        self._keep[hash_index] = (table, d_wkv, d_qk)
        _check(lib().engram_ctx_add_layer(self.h, hash_index, ctypes.byref(table.c),
                                          _ptr(d_wkv), _ptr(d_qk)))

    def set_wkv_q2k(self, hash_index, d_wq):
        """Registers (or, with None, drops) the layer's wkv as Q2_K blocks."""
        table, wkv, qk = self._keep[hash_index][:3]
        N, K = self.dim * (self.hc + 1), self.cols * self.head_dim
        _need(d_wq, "wkv_q2k", N * (K // 256) * 84)
        self._keep[hash_index] = (table, wkv, qk, d_wq)
        _check(lib().engram_ctx_set_wkv_q2k(self.h, hash_index, _ptr(d_wq)))

    def reset(self, stream=None):
        _check(lib().engram_reset(self.h, _stream(stream)))

    def forward(self, hash_index, d_ids, T, d_h, stream=None):
        M = self.batch * int(T)
        _need(d_ids, "ids", 4 * M)
        _need(d_h, "h", 4 * M * self.hc * self.dim)
        _check(lib().engram_forward(self.h, hash_index, _ptr(d_ids), int(T), _ptr(d_h),
                                    _stream(stream)))

    def check(self, stream=None):
        _check(lib().engram_check(self.h, _stream(stream)))

    @property
    def position(self):
        return lib().engram_position(self.h)

    def buffers(self):
        """(row_ids, rows, kv, err) device addresses."""
        ptrs = [ctypes.c_void_p() for _ in range(4)]
        _check(lib().engram_ctx_buffers(self.h, *[ctypes.byref(q) for q in ptrs]))
        return tuple(q.value for q in ptrs)

    def views(self, T):
        """torch views of the workspace for a call of T tokens a sequence
        (M = batch*T): row ids [M, nl, cols] int64, rows [M, cols*head_dim]
        bf16 bits (int16), kv [M, dim*(hc+1)] (int16)."""
        import torch
        ws = self.workspace
        base = ws.data_ptr()
        rid, rows, kv, _ = self.buffers()

        def view(addr, n, dtype, shape):
            size = torch.empty(0, dtype=dtype).element_size()
            off = addr - base
            return ws[off:off + n * size].view(dtype).view(*shape)

        K, N = self.cols * self.head_dim, self.dim * (self.hc + 1)
        M = self.batch * T
        return (view(rid, M * self.nl * self.cols, torch.int64, (M, self.nl, self.cols)),
                view(rows, M * K, torch.int16, (M, K)),
                view(kv, M * N, torch.int16, (M, N)))

    def set_fused_decode(self, on: bool):
        _check(lib().engram_ctx_set_fused_decode(self.h, 1 if on else 0))

    def set_timing(self, on: bool):
        _check(lib().engram_ctx_set_timing(self.h, 1 if on else 0))

    def history(self):
        """The hasher's history rows, a view of the workspace: [batch, max_seq]
        int64 compressed ids (what a checkpoint of the sequence holds)."""
        import torch
        n = self.batch * int(self.cfg.max_seq)
        return self.workspace[:8 * n].view(torch.int64).view(self.batch, -1)

    def set_position(self, pos, stream=None):
        """Resume at pos over history rows the caller restored into the
        workspace (engram_ctx_set_position)."""
        _check(lib().engram_ctx_set_position(self.h, int(pos), _stream(stream)))

    def set_graph_mode(self, on: bool, stream=None):
        """Single-token steps read their position from the device, so their
        launches can be captured once and replayed (engram_ctx_set_graph_mode)."""
        _check(lib().engram_ctx_set_graph_mode(self.h, 1 if on else 0, _stream(stream)))

    def timing(self):
        ms = (ctypes.c_double * 4)()
        n = (ctypes.c_int64 * 4)()
        _check(lib().engram_ctx_timing(self.h, ms, n))
        return {STAGES[i]: (ms[i], n[i]) for i in range(4)}

    def close(self):
        if getattr(self, "h", None):
            lib().engram_ctx_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
