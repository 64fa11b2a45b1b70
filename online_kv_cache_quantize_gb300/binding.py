"""ctypes binding of libtq (include/tq.h): the same entry-point names, argument
marshalling only. Every step of the hot path runs in the library's CUDA
kernels; PyTorch supplies device memory and streams.

The library is loaded on first use from this package directory. If it is
missing, every call raises: there is no CPU fallback.
"""

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libtq.so")
_lib = None

TQ_OK = 0
TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED = 1, 2
TQ_ERR_TIMEOUT = 6
TQ_ERR_WORKSPACE = 7
TQ_ROT_DENSE_QR, TQ_ROT_RHT = 0, 1
TQ_MSE, TQ_PROD, TQ_POLAR = 0, 1, 2
TQ_F32, TQ_BF16, TQ_F16 = 0, 1, 2

ROT_KINDS = {"dense": TQ_ROT_DENSE_QR, "rht": TQ_ROT_RHT}
MODES = {"mse": TQ_MSE, "prod": TQ_PROD, "polar": TQ_POLAR}


class TQError(RuntimeError):
    def __init__(self, status, where, message):
        super().__init__(f"{where}: {status_name(status)} ({message})")
        self.status = status


class tq_cache(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("bits", ctypes.c_int), ("d", ctypes.c_int), ("m", ctypes.c_int),
                ("rows", ctypes.c_int64), ("capacity", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("signs", ctypes.c_void_p),
                ("norm", ctypes.c_void_p), ("rnorm", ctypes.c_void_p), ("bits2", ctypes.c_int)]


class tq_quant_args(ctypes.Structure):
    _fields_ = [("cache", tq_cache), ("rot", ctypes.c_void_p), ("qjl", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("x_dtype", ctypes.c_int), ("x_stride", ctypes.c_int64),
                ("n", ctypes.c_int64), ("dst_slot", ctypes.c_void_p), ("append_pos", ctypes.c_void_p),
                ("heads", ctypes.c_int), ("slot0", ctypes.c_int64)]


class tq_decode_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_dtype", ctypes.c_int),
                ("batch", ctypes.c_int), ("hq", ctypes.c_int), ("hkv", ctypes.c_int), ("d", ctypes.c_int),
                ("seq_lens", ctypes.c_void_p), ("max_seq_len", ctypes.c_int),
                ("gqa_map", ctypes.c_void_p), ("rot", ctypes.c_void_p), ("qjl", ctypes.c_void_p),
                ("k", tq_cache), ("v", tq_cache), ("scale", ctypes.c_float), ("n_splits", ctypes.c_int),
                ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int), ("logits", ctypes.c_void_p),
                ("scan_begin", ctypes.c_void_p), ("scan_end", ctypes.c_void_p)]


class tq_step_args(ctypes.Structure):
    _fields_ = [("attn", tq_decode_args), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
                ("new_dtype", ctypes.c_int), ("append_pos", ctypes.c_void_p)]


class tq_prefill_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_dtype", ctypes.c_int),
                ("batch", ctypes.c_int), ("chunk", ctypes.c_int), ("hq", ctypes.c_int), ("hkv", ctypes.c_int),
                ("d", ctypes.c_int), ("q_start", ctypes.c_void_p), ("max_context", ctypes.c_int),
                ("gqa_map", ctypes.c_void_p), ("rot", ctypes.c_void_p), ("qjl", ctypes.c_void_p), ("k", tq_cache), ("v", tq_cache),
                ("scale", ctypes.c_float), ("n_splits", ctypes.c_int), ("out", ctypes.c_void_p),
                ("out_dtype", ctypes.c_int), ("scan_begin", ctypes.c_void_p), ("scan_end", ctypes.c_void_p)]


class tq_topk_args(ctypes.Structure):
    _fields_ = [("queries", ctypes.c_void_p), ("nq", ctypes.c_int), ("d", ctypes.c_int),
                ("rot", ctypes.c_void_p), ("qjl", ctypes.c_void_p), ("db", tq_cache),
                ("n_db", ctypes.c_int64), ("k", ctypes.c_int), ("ids", ctypes.c_void_p),
                ("scores", ctypes.c_void_p)]


class tq_view(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int), ("sinks", ctypes.c_int), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int), ("n_pages", ctypes.c_int)]


class tq_decode_view_args(ctypes.Structure):
    _fields_ = [("attn", tq_decode_args), ("view", tq_view)]


class tq_step_view_args(ctypes.Structure):
    _fields_ = [("step", tq_step_args), ("view", tq_view)]


class tq_prefill_view_args(ctypes.Structure):
    _fields_ = [("attn", tq_prefill_args), ("view", tq_view)]


class tq_page_pool(ctypes.Structure):
    _fields_ = [("k", tq_cache), ("v", tq_cache), ("hkv", ctypes.c_int), ("n_pages", ctypes.c_int),
                ("refs", ctypes.c_void_p)]


class tq_page_table(ctypes.Structure):
    _fields_ = [("entries", ctypes.c_void_p), ("stride", ctypes.c_int64), ("rows", ctypes.c_int),
                ("max_pages", ctypes.c_int)]


class tq_pages_reserve_args(ctypes.Structure):
    _fields_ = [("pool", tq_page_pool), ("table", tq_page_table), ("lengths", ctypes.c_void_p),
                ("add", ctypes.c_void_p), ("add_all", ctypes.c_int), ("shortage", ctypes.c_void_p),
                ("granted", ctypes.c_void_p)]


class tq_pages_trim_args(ctypes.Structure):
    _fields_ = [("pool", tq_page_pool), ("table", tq_page_table), ("lengths", ctypes.c_void_p),
                ("window", ctypes.c_int), ("sinks", ctypes.c_int)]


class tq_pages_fork_args(ctypes.Structure):
    _fields_ = [("pool", tq_page_pool), ("src", tq_page_table), ("dst", tq_page_table),
                ("parent", ctypes.c_void_p), ("src_lengths", ctypes.c_void_p), ("dst_lengths", ctypes.c_void_p),
                ("keep_src", ctypes.c_int), ("shortage", ctypes.c_void_p)]


class tq_pages_copy_args(ctypes.Structure):
    _fields_ = [("src", tq_page_pool), ("dst", tq_page_pool), ("src_pages", ctypes.c_void_p),
                ("dst_pages", ctypes.c_void_p), ("n", ctypes.c_int)]


TQ_MAX_PAGE_TABLES = 4


class tq_pages_compact_args(ctypes.Structure):
    _fields_ = [("src", tq_page_pool), ("dst", tq_page_pool), ("src_tables", tq_page_table * TQ_MAX_PAGE_TABLES),
                ("dst_tables", tq_page_table * TQ_MAX_PAGE_TABLES), ("n_tables", ctypes.c_int),
                ("live", ctypes.c_void_p)]


_STATUS = ctypes.c_int
_SIGS = {
    "tq_status_string": (ctypes.c_char_p, [_STATUS]),
    "tq_last_error": (ctypes.c_char_p, []),
    "tq_abi_struct_size": (ctypes.c_size_t, [ctypes.c_char_p]),
    "tq_random_stream": (_STATUS, [ctypes.c_uint64, ctypes.c_uint64, ctypes.c_int64, ctypes.c_void_p]),
    "tq_make_rotation": (_STATUS, [ctypes.c_uint64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)]),
    "tq_rotation_get": (_STATUS, [ctypes.c_void_p, ctypes.c_void_p]),
    "tq_rotation_info": (_STATUS, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tq_rotation_to_device": (_STATUS, [ctypes.c_void_p]),
    "tq_free_rotation": (_STATUS, [ctypes.c_void_p]),
    "tq_make_qjl": (_STATUS, [ctypes.c_uint64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)]),
    "tq_qjl_get": (_STATUS, [ctypes.c_void_p, ctypes.c_void_p]),
    "tq_qjl_to_device": (_STATUS, [ctypes.c_void_p]),
    "tq_free_qjl": (_STATUS, [ctypes.c_void_p]),
    "tq_codebook": (_STATUS, [ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "tq_code_bytes": (ctypes.c_int, [ctypes.c_int, ctypes.c_int]),
    "tq_code_bytes2": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "tq_sign_bytes": (ctypes.c_int, [ctypes.c_int]),
    "tq_polar_code_bytes": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "tq_polar_codebook": (_STATUS, [ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "tq_quantize_kv": (_STATUS, [ctypes.POINTER(tq_quant_args), ctypes.c_void_p]),
    "tq_attn_decode_workspace": (ctypes.c_size_t, [ctypes.POINTER(tq_decode_args)]),
    "tq_attn_decode": (_STATUS, [ctypes.POINTER(tq_decode_args), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "tq_attn_prefill_workspace": (ctypes.c_size_t, [ctypes.POINTER(tq_prefill_args)]),
    "tq_attn_prefill": (_STATUS, [ctypes.POINTER(tq_prefill_args), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "tq_attn_decode_static": (_STATUS, [ctypes.POINTER(tq_decode_args), ctypes.c_void_p]),
    "tq_score_topk_workspace": (ctypes.c_size_t, [ctypes.POINTER(tq_topk_args)]),
    "tq_score_topk": (_STATUS, [ctypes.POINTER(tq_topk_args), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "tq_decode_step_workspace": (ctypes.c_size_t, [ctypes.POINTER(tq_step_args)]),
    "tq_decode_step": (_STATUS, [ctypes.POINTER(tq_step_args), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "tq_attn_decode_view_workspace": (ctypes.c_size_t, [ctypes.POINTER(tq_decode_view_args)]),
    "tq_attn_decode_view": (_STATUS, [ctypes.POINTER(tq_decode_view_args), ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_void_p]),
    "tq_decode_step_view_workspace": (ctypes.c_size_t, [ctypes.POINTER(tq_step_view_args)]),
    "tq_decode_step_view": (_STATUS, [ctypes.POINTER(tq_step_view_args), ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_void_p]),
    "tq_attn_prefill_view_workspace": (ctypes.c_size_t, [ctypes.POINTER(tq_prefill_view_args)]),
    "tq_attn_prefill_view": (_STATUS, [ctypes.POINTER(tq_prefill_view_args), ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "tq_pages_workspace": (ctypes.c_size_t, [ctypes.POINTER(tq_page_pool), ctypes.c_int]),
    "tq_pages_reserve": (_STATUS, [ctypes.POINTER(tq_pages_reserve_args), ctypes.c_void_p, ctypes.c_size_t,
                                   ctypes.c_void_p]),
    "tq_pages_trim": (_STATUS, [ctypes.POINTER(tq_pages_trim_args), ctypes.c_void_p]),
    "tq_pages_fork": (_STATUS, [ctypes.POINTER(tq_pages_fork_args), ctypes.c_void_p, ctypes.c_size_t,
                                ctypes.c_void_p]),
    "tq_pages_copy": (_STATUS, [ctypes.POINTER(tq_pages_copy_args), ctypes.c_void_p]),
    "tq_pages_compact": (_STATUS, [ctypes.POINTER(tq_pages_compact_args), ctypes.c_void_p, ctypes.c_size_t,
                                   ctypes.c_void_p]),
    "tq_topk_force_simt": (ctypes.c_int, [ctypes.c_int]),
    "tq_quantize_force_mma_sync": (ctypes.c_int, [ctypes.c_int]),
    "tq_prefill_force_mma_sync": (ctypes.c_int, [ctypes.c_int]),
    "tq_device_errors": (_STATUS, [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]),
    "tq_selftest_bounded_wait": (_STATUS, [ctypes.c_uint32, ctypes.c_void_p]),
    "tq_selftest_umma_gemm": (_STATUS, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p]),
    "tq_selftest_umma_gemm_tmem_a": (_STATUS, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p]),
}

EXPORTED = tuple(_SIGS)


def lib_path():
    return _LIB_PATH


def load():
    """Load libtq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"libtq.so not built at {_LIB_PATH}; run online_kv_cache_quantize_gb300.build")
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    for name, cls in (("tq_cache", tq_cache), ("tq_quant_args", tq_quant_args),
                      ("tq_decode_args", tq_decode_args), ("tq_topk_args", tq_topk_args),
                      ("tq_step_args", tq_step_args), ("tq_prefill_args", tq_prefill_args),
                      ("tq_view", tq_view), ("tq_decode_view_args", tq_decode_view_args),
                      ("tq_step_view_args", tq_step_view_args), ("tq_prefill_view_args", tq_prefill_view_args),
                      ("tq_page_pool", tq_page_pool), ("tq_page_table", tq_page_table),
                      ("tq_pages_reserve_args", tq_pages_reserve_args), ("tq_pages_trim_args", tq_pages_trim_args),
                      ("tq_pages_fork_args", tq_pages_fork_args), ("tq_pages_copy_args", tq_pages_copy_args),
                      ("tq_pages_compact_args", tq_pages_compact_args)):
        if lib.tq_abi_struct_size(name.encode()) != ctypes.sizeof(cls):
            raise RuntimeError(f"struct {name} layout differs between libtq.so and the binding")
    _lib = lib
    return lib


def status_name(s):
    return load().tq_status_string(s).decode()


def _check(status, where):
    if status != TQ_OK:
        raise TQError(status, where, load().tq_last_error().decode())


# ---------------------------------------------------------------- set-up ---
def tq_random_stream(seed, count, start=0):
    out = np.empty(count, dtype=np.uint64)
    _check(load().tq_random_stream(seed, start, count, out.ctypes.data), "tq_random_stream")
    return out


class Rotation:
    """Owns a tq_rotation handle."""

    def __init__(self, handle, d, kind):
        self.handle, self.d, self.kind = handle, d, kind

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.tq_free_rotation(self.handle)
            self.handle = None


class QJL:
    """Owns a tq_qjl handle."""

    def __init__(self, handle, m, d):
        self.handle, self.m, self.d = handle, m, d

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.tq_free_qjl(self.handle)
            self.handle = None


def tq_make_rotation(seed, d, kind="dense"):
    h = ctypes.c_void_p()
    k = ROT_KINDS.get(kind, kind)
    _check(load().tq_make_rotation(seed, d, k, ctypes.byref(h)), "tq_make_rotation")
    return Rotation(h.value, d, k)


def tq_rotation_get(rot):
    out = np.empty((rot.d, rot.d), dtype=np.float64)
    _check(load().tq_rotation_get(rot.handle, out.ctypes.data), "tq_rotation_get")
    return out


def tq_rotation_to_device(rot):
    _check(load().tq_rotation_to_device(rot.handle), "tq_rotation_to_device")
    return rot


def tq_make_qjl(seed, m, d):
    h = ctypes.c_void_p()
    _check(load().tq_make_qjl(seed, m, d, ctypes.byref(h)), "tq_make_qjl")
    return QJL(h.value, m, d)


def tq_qjl_get(qjl):
    out = np.empty((qjl.m, qjl.d), dtype=np.float64)
    _check(load().tq_qjl_get(qjl.handle, out.ctypes.data), "tq_qjl_get")
    return out


def tq_qjl_to_device(qjl):
    _check(load().tq_qjl_to_device(qjl.handle), "tq_qjl_to_device")
    return qjl


def tq_codebook(d, bits):
    c = np.empty(1 << bits, dtype=np.float64)
    t = np.empty((1 << bits) - 1, dtype=np.float64)
    _check(load().tq_codebook(d, bits, c.ctypes.data, t.ctypes.data), "tq_codebook")
    return c, t


def tq_code_bytes(d, code_bits):
    return load().tq_code_bytes(d, code_bits)


def tq_sign_bytes(m):
    return load().tq_sign_bytes(m)


def tq_polar_code_bytes(d, bits1, bits2):
    return load().tq_polar_code_bytes(d, bits1, bits2)


def tq_polar_codebook(level, bits):
    c = np.empty(1 << bits, dtype=np.float64)
    t = np.empty((1 << bits) - 1, dtype=np.float64)
    _check(load().tq_polar_codebook(level, bits, c.ctypes.data, t.ctypes.data), "tq_polar_codebook")
    return c, t


# ------------------------------------------------------- cache planes ---
class Cache:
    """Device planes of a packed cache (torch tensors owned by this object)."""

    def __init__(self, mode, bits, d, rows, capacity, m=None, device="cuda", bits2=None):
        """bits2: the second channel group's bits of a fractional-rate cache
        (coordinates with i % 16 >= 8), None for one width; for a PolarQuant
        cache ("polar") the bits of the angles above level 1 (required)."""
        import torch

        self.mode = MODES.get(mode, mode)
        self.bits, self.d, self.rows, self.capacity = bits, d, rows, capacity
        if self.mode == TQ_POLAR:
            if not bits2:
                raise ValueError("a PolarQuant cache needs bits2 (the bits of the angles above level 1)")
            self.bits2 = bits2
        else:
            self.bits2 = bits2 if bits2 and bits2 != bits else None
        self.m = (m if m is not None else d) if self.mode == TQ_PROD else 0
        cb = bits - 1 if self.mode == TQ_PROD else bits
        self.code_bits = cb
        n = rows * capacity
        if self.mode == TQ_POLAR:
            self.code_stride = tq_polar_code_bytes(d, bits, bits2)
        elif self.bits2 is None:
            self.code_stride = tq_code_bytes(d, cb)
        else:
            self.code_stride = load().tq_code_bytes2(d, cb, self.bits2 - 1 if self.mode == TQ_PROD else self.bits2)
        self.codes = torch.zeros((n, self.code_stride), dtype=torch.uint8, device=device)
        self.norm = torch.zeros(n, dtype=torch.int16, device=device)
        if self.mode == TQ_PROD:
            self.sign_stride = tq_sign_bytes(self.m)
            self.signs = torch.zeros((n, self.sign_stride), dtype=torch.uint8, device=device)
            self.rnorm = torch.zeros(n, dtype=torch.int16, device=device)
        else:
            self.sign_stride = 0
            self.signs = None
            self.rnorm = None

    def struct(self):
        return tq_cache(self.mode, self.bits, self.d, self.m, self.rows, self.capacity,
                        self.codes.data_ptr(), self.signs.data_ptr() if self.signs is not None else None,
                        self.norm.data_ptr(), self.rnorm.data_ptr() if self.rnorm is not None else None,
                        self.bits2 or 0)

    def bytes_per_slot(self):
        return self.code_stride + 2 + (self.sign_stride + 2 if self.mode == TQ_PROD else 0)


def _dtype_code(t):
    import torch

    return {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}[t.dtype]


_current_stream = None  # () -> the current device's current stream, as an address


def _stream_ptr(stream):
    if stream is not None:
        return stream.cuda_stream
    global _current_stream
    if _current_stream is None:
        _current_stream = _stream_getter()
    return _current_stream()


def _stream_getter():
    """torch.cuda.current_stream() makes a Stream object each time (3 us); the address alone is enough here."""
    import torch

    torch.cuda.current_stream()  # initialises CUDA, or raises
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(device())


# ------------------------------------------------------------- hot path ---
def tq_quantize_kv(cache, rot, x, qjl=None, slot0=0, dst_slot=None, append_pos=None, heads=1, stream=None):
    """Quantize rows of x (device [n, >=d], f32 or bf16) into `cache`."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit inner stride")
    a = tq_quant_args()
    a.cache = cache.struct()
    a.rot = rot.handle
    a.qjl = qjl.handle if qjl is not None else None
    a.x = x.data_ptr()
    a.x_dtype = _dtype_code(x)
    a.x_stride = x.stride(0)
    a.n = x.shape[0]
    a.dst_slot = dst_slot.data_ptr() if dst_slot is not None else None
    a.append_pos = append_pos.data_ptr() if append_pos is not None else None
    a.heads = heads
    a.slot0 = slot0
    _check(load().tq_quantize_kv(ctypes.byref(a), _stream_ptr(stream)), "tq_quantize_kv")


def _decode_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, scale=0.0, n_splits=0,
                   gqa_map=None, logits=None, hkv=None):
    b, hq, d = q.shape
    a = tq_decode_args()
    a.q = q.data_ptr()
    a.q_dtype = _dtype_code(q)
    a.batch, a.hq, a.hkv, a.d = b, hq, hkv if hkv is not None else kcache.rows // b, d
    a.seq_lens = seq_lens.data_ptr()
    a.max_seq_len = max_seq_len
    keep = None
    if gqa_map is not None:
        keep = np.ascontiguousarray(gqa_map, dtype=np.int32)
        a.gqa_map = keep.ctypes.data
    a.rot = rot.handle
    a.qjl = qjl.handle if qjl is not None else None
    a.k = kcache.struct()
    a.v = vcache.struct()
    a.scale = scale
    a.n_splits = n_splits
    a.out = out.data_ptr()
    a.out_dtype = _dtype_code(out)
    a.logits = logits.data_ptr() if logits is not None else None
    return a, keep


def tq_attn_decode_workspace(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, **kw):
    a, _keep = _decode_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, **kw)
    return load().tq_attn_decode_workspace(ctypes.byref(a))


def tq_attn_decode(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, workspace, stream=None, **kw):
    """Decode attention over the packed caches; writes `out` (and `logits` if given)."""
    a, _keep = _decode_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, **kw)
    _check(load().tq_attn_decode(ctypes.byref(a), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 _stream_ptr(stream)), "tq_attn_decode")


def _prefill_struct(q, kcache, vcache, q_start, max_context, rot, qjl, out, scale=0.0, n_splits=0, gqa_map=None,
                    scan_events=None, hkv=None):
    b, c, hq, d = q.shape
    a = tq_prefill_args()
    keep = None
    if gqa_map is not None:
        keep = np.ascontiguousarray(gqa_map, dtype=np.int32)
        a.gqa_map = keep.ctypes.data
    a.q = q.data_ptr()
    a.q_dtype = _dtype_code(q)
    a.batch, a.chunk, a.hq, a.hkv, a.d = b, c, hq, hkv if hkv is not None else kcache.rows // b, d
    a.q_start = q_start.data_ptr()
    a.max_context = max_context
    a.rot = rot.handle
    a.qjl = qjl.handle if qjl is not None else None
    a.k = kcache.struct()
    a.v = vcache.struct()
    a.scale = scale
    a.n_splits = n_splits
    a.out = out.data_ptr()
    a.out_dtype = _dtype_code(out)
    if scan_events is not None:  # (begin, end) torch.cuda.Event pair, recorded around the scan kernel
        a.scan_begin = scan_events[0].cuda_event
        a.scan_end = scan_events[1].cuda_event
    return a, keep


def tq_attn_prefill_workspace(q, kcache, vcache, q_start, max_context, rot, qjl, out, **kw):
    a, _keep = _prefill_struct(q, kcache, vcache, q_start, max_context, rot, qjl, out, **kw)
    return load().tq_attn_prefill_workspace(ctypes.byref(a))


def tq_attn_prefill(q, kcache, vcache, q_start, max_context, rot, qjl, out, workspace, stream=None, **kw):
    """Chunked-prefill attention: q [batch][chunk][hq][d], the chunk of each
    sequence starting at position q_start[b] (device int32) and already
    quantized into the caches; writes out [batch][chunk][hq][d]."""
    a, _keep = _prefill_struct(q, kcache, vcache, q_start, max_context, rot, qjl, out, **kw)
    _check(load().tq_attn_prefill(ctypes.byref(a), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream_ptr(stream)), "tq_attn_prefill")


def tq_attn_decode_static(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, stream=None, **kw):
    """tq_attn_decode without a workspace: for callers that may not allocate
    device memory; its scratch is an array inside the library (see tq.h)."""
    a, _keep = _decode_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, **kw)
    _check(load().tq_attn_decode_static(ctypes.byref(a), _stream_ptr(stream)), "tq_attn_decode_static")


def _step_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos, **kw):
    attn, keep = _decode_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, **kw)
    a = tq_step_args()
    a.attn = attn
    a.k_new = k_new.data_ptr()
    a.v_new = v_new.data_ptr()
    if k_new.dtype != v_new.dtype:
        raise ValueError("k_new and v_new must have the same dtype")
    a.new_dtype = _dtype_code(k_new)
    a.append_pos = append_pos.data_ptr()
    return a, keep


def tq_decode_step_workspace(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos, **kw):
    a, _keep = _step_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos, **kw)
    return load().tq_decode_step_workspace(ctypes.byref(a))


def tq_decode_step(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos, workspace,
                   stream=None, **kw):
    """Append the new token's K and V (rows b*hkv + h of k_new / v_new at slot
    append_pos[b]) and run decode attention, in one call."""
    a, _keep = _step_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos, **kw)
    _check(load().tq_decode_step(ctypes.byref(a), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 _stream_ptr(stream)), "tq_decode_step")


# ------------------------------------------- windowed and paged attention ---
def _int32_ptr(t, what, n=None):
    """Device pointer of a contiguous int32 tensor (None stays None)."""
    import torch

    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor")
    if n is not None and t.numel() < n:
        raise ValueError(f"{what} must hold {n} values")
    return t.data_ptr()


def _table_check(t, what):
    import torch

    if t.dtype != torch.int32 or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be a 2-D int32 tensor with unit inner stride")


def _int_check(x, what):
    """The C structs hold int32: a larger number would be cut to its low bits."""
    if not -2**31 <= x < 2**31:
        raise ValueError(f"{what} must fit 32 bits")
    return x


def _device_check(home, **tensors):
    """Every tensor of a call lies on the GPU that `home` lies on, and the call
    goes to that GPU."""
    import torch

    for what, t in tensors.items():
        if t is not None and t.device != home.device:
            raise ValueError(f"{what} is on {t.device}, the caches are on {home.device}")
    if home.device.type != "cuda":
        raise ValueError("the caches must be on a GPU")
    if torch.cuda.current_device() != home.device.index:
        raise ValueError(f"the caches are on {home.device}, the current device is cuda:{torch.cuda.current_device()}")


def _dense_check(t, what, n, dtypes=None):
    """A contiguous tensor of n values (the kernels know no strides)."""
    import torch

    names = dtypes or (torch.float32, torch.bfloat16)
    if t.dtype not in names:
        raise ValueError(f"{what} must be of {' or '.join(str(x) for x in names)}")
    if not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{what} must be contiguous and hold {n} values")


def _attend_check(view, kcache, vcache, q, pos, pos_name, out, gqa_map=None, logits=None, max_seq_len=0, rows=None,
                  **_):
    """The tensors of a windowed / paged attention call, before their addresses go to the library."""
    import torch

    batch, hq, d = q.shape[0], q.shape[-2], q.shape[-1]
    _dense_check(q, "q", q.numel())
    _dense_check(out, "out", q.numel())
    _int32_ptr(pos, pos_name, batch)
    if gqa_map is not None and len(gqa_map) != hq:
        raise ValueError("gqa_map must have an entry per query head")
    if logits is not None:
        _dense_check(logits, "logits", batch * hq * max_seq_len if max_seq_len > 0 else logits.numel(), (torch.float32,))
    k_new, v_new, append_pos = rows or (None, None, None)
    if rows:
        n = batch * view.hkv(kcache, batch) * d
        _dense_check(k_new, "k_new", n)
        _dense_check(v_new, "v_new", n, (k_new.dtype,))
        _int32_ptr(append_pos, "append_pos", batch)
    _device_check(kcache.codes, vcache=vcache.codes, q=q, out=out, logits=logits, page_table=view.page_table, k_new=k_new,
                  v_new=v_new, append_pos=append_pos, **{pos_name: pos})


class View:
    """What an attention call sees of each sequence (tq_view): window (0: every
    token) and sinks, and, for a paged cache, its page table (device int32
    [batch, max_pages]) and the pool's page count."""

    def __init__(self, window=0, sinks=0, page_table=None, n_pages=0):
        if page_table is not None:
            _table_check(page_table, "page_table")
        self.window, self.sinks, self.n_pages = (_int_check(x, w) for x, w in ((window, "window"), (sinks, "sinks"),
                                                                              (n_pages, "n_pages")))
        self.page_table = page_table

    def struct(self):
        t = self.page_table
        if t is None:
            return tq_view(self.window, self.sinks, None, 0, 0, self.n_pages)
        return tq_view(self.window, self.sinks, t.data_ptr(), t.stride(0), t.shape[1], self.n_pages)

    def hkv(self, cache, batch):
        """KV heads of a cache seen this way."""
        rows = self.n_pages if self.page_table is not None else batch
        if rows < 1 or cache.rows % rows:
            raise ValueError("the cache's rows are not a multiple of the view's pages (or of the batch)")
        if self.page_table is not None and self.page_table.shape[0] != batch:
            raise ValueError("page_table must have a row per sequence")
        return cache.rows // rows


class BoundCall:
    """A hot-path call with its argument struct formed once: call it as often
    as its tensors stay where they are (their contents may change). Returned
    by `prepare`; holds references to the tensors."""

    def __init__(self, name, struct, workspace, keep):
        self._fn, self._name, self._a, self._keep = getattr(load(), name), name, struct, (workspace, keep)
        self._args = (ctypes.byref(struct),)
        if workspace is not None:
            if not workspace.is_contiguous():
                raise ValueError("the workspace must be contiguous")
            self._args += (ctypes.c_void_p(workspace.data_ptr()),
                           ctypes.c_size_t(workspace.numel() * workspace.element_size()))

    def __call__(self, stream=None):
        st = self._fn(*self._args, _stream_ptr(stream))
        if st != TQ_OK:
            _check(st, self._name)


_BUILDERS = {}


def _bindable(name):
    """Registers the function that forms the call of entry point `name`."""
    def add(build):
        def call(*args, stream=None, **kw):
            build(*args, **kw)(stream)

        call.__name__, call.__doc__ = name, build.__doc__
        _BUILDERS[call] = build
        return call
    return add


def prepare(fn, *args, **kw):
    """A BoundCall of one of the windowed / paged / page functions below with
    these arguments (all but `stream`, which its calls take)."""
    if fn not in _BUILDERS:
        raise ValueError("prepare takes the *_view and tq_pages_* functions")
    return _BUILDERS[fn](*args, **kw)


def _decode_view_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, view, **kw):
    _attend_check(view, kcache, vcache, q, seq_lens, "seq_lens", out, max_seq_len=max_seq_len, **kw)
    attn, keep = _decode_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out,
                                hkv=view.hkv(kcache, q.shape[0]), **kw)
    return tq_decode_view_args(attn, view.struct()), (keep, q, kcache, vcache, seq_lens, rot, qjl, out, view, kw)


def tq_attn_decode_view_workspace(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, view, **kw):
    a, _keep = _decode_view_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, view, **kw)
    return load().tq_attn_decode_view_workspace(ctypes.byref(a))


@_bindable("tq_attn_decode_view")
def tq_attn_decode_view(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, workspace, view, **kw):
    """tq_attn_decode over the tokens `view` leaves visible, of contiguous or
    paged caches (a paged cache has n_pages * hkv rows)."""
    a, keep = _decode_view_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, view, **kw)
    _device_check(kcache.codes, workspace=workspace)
    return BoundCall("tq_attn_decode_view", a, workspace, keep)


def _step_view_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos, view, **kw):
    _attend_check(view, kcache, vcache, q, seq_lens, "seq_lens", out, max_seq_len=max_seq_len,
                  rows=(k_new, v_new, append_pos), **kw)
    step, keep = _step_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos,
                              hkv=view.hkv(kcache, q.shape[0]), **kw)
    return tq_step_view_args(step, view.struct()), (keep, q, kcache, vcache, seq_lens, rot, qjl, out, k_new, v_new,
                                                    append_pos, view, kw)


def tq_decode_step_view_workspace(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos,
                                  view, **kw):
    a, _keep = _step_view_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos,
                                 view, **kw)
    return load().tq_decode_step_view_workspace(ctypes.byref(a))


@_bindable("tq_decode_step_view")
def tq_decode_step_view(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos, workspace,
                        view, **kw):
    """tq_decode_step over the tokens `view` leaves visible; the new token of
    sequence b goes to position append_pos[b] through the page table."""
    a, keep = _step_view_struct(q, kcache, vcache, seq_lens, max_seq_len, rot, qjl, out, k_new, v_new, append_pos,
                                view, **kw)
    _device_check(kcache.codes, workspace=workspace)
    return BoundCall("tq_decode_step_view", a, workspace, keep)


def _prefill_view_struct(q, kcache, vcache, q_start, max_context, rot, qjl, out, view, **kw):
    _attend_check(view, kcache, vcache, q, q_start, "q_start", out, **kw)
    attn, keep = _prefill_struct(q, kcache, vcache, q_start, max_context, rot, qjl, out,
                                 hkv=view.hkv(kcache, q.shape[0]), **kw)
    return tq_prefill_view_args(attn, view.struct()), (keep, q, kcache, vcache, q_start, rot, qjl, out, view, kw)


def tq_attn_prefill_view_workspace(q, kcache, vcache, q_start, max_context, rot, qjl, out, view, **kw):
    a, _keep = _prefill_view_struct(q, kcache, vcache, q_start, max_context, rot, qjl, out, view, **kw)
    return load().tq_attn_prefill_view_workspace(ctypes.byref(a))


@_bindable("tq_attn_prefill_view")
def tq_attn_prefill_view(q, kcache, vcache, q_start, max_context, rot, qjl, out, workspace, view, **kw):
    """tq_attn_prefill over the tokens `view` leaves visible to each query."""
    a, keep = _prefill_view_struct(q, kcache, vcache, q_start, max_context, rot, qjl, out, view, **kw)
    _device_check(kcache.codes, workspace=workspace)
    return BoundCall("tq_attn_prefill_view", a, workspace, keep)


# ------------------------------------------------------------ page calls ---
class PagePool:
    """A key and a value Cache as a pool of pages (tq_page_pool): n_pages pages
    of `capacity` tokens and hkv heads, and the device counts of their holders
    (refs, zeros unless given)."""

    def __init__(self, kcache, vcache, hkv, refs=None):
        import torch

        if kcache.rows % hkv:
            raise ValueError("the cache's rows must be a multiple of hkv")
        self.k, self.v, self.hkv, self.n_pages, self.page = kcache, vcache, hkv, kcache.rows // hkv, kcache.capacity
        self.refs = refs if refs is not None else torch.zeros(self.n_pages, dtype=torch.int32,
                                                              device=kcache.codes.device)
        _int32_ptr(self.refs, "refs", self.n_pages)
        if self.refs.device != kcache.codes.device or vcache.codes.device != kcache.codes.device:
            raise ValueError("the caches and refs must be on one device")

    def table(self, rows, max_pages):
        """An empty page table (every entry -1)."""
        import torch

        return torch.full((rows, max_pages), -1, dtype=torch.int32, device=self.refs.device)

    def struct(self):
        return tq_page_pool(self.k.struct(), self.v.struct(), self.hkv, self.n_pages, self.refs.data_ptr())


def _table_struct(t):
    _table_check(t, "a page table")
    return tq_page_table(t.data_ptr(), t.stride(0), t.shape[0], t.shape[1])


def tq_pages_workspace(pool, rows):
    """Workspace bytes of the page calls on `pool` for tables of at most `rows` rows."""
    a = pool.struct()
    return load().tq_pages_workspace(ctypes.byref(a), rows)


@_bindable("tq_pages_reserve")
def tq_pages_reserve(pool, table, lengths, add, workspace, shortage=None, granted=None):
    """Pages for the `add` tokens (an int, or device int32 per row) behind each
    row's lengths[b] tokens; a half-filled last page that other rows hold too is
    replaced by a copy. granted (device int32 per row): how many of these tokens
    lie in pages the row holds, from the first on; below 0 the tokens that the
    row lost with its last page."""
    a = tq_pages_reserve_args(pool.struct(), _table_struct(table), _int32_ptr(lengths, "lengths", table.shape[0]))
    if isinstance(add, int):
        a.add_all = _int_check(add, "add")
    else:
        a.add = _int32_ptr(add, "add", table.shape[0])
    a.shortage = _int32_ptr(shortage, "shortage", 1)
    a.granted = _int32_ptr(granted, "granted", table.shape[0])
    _device_check(pool.refs, table=table, lengths=lengths, add=None if isinstance(add, int) else add, shortage=shortage,
                  granted=granted, workspace=workspace)
    return BoundCall("tq_pages_reserve", a, workspace, (pool, table, lengths, add, shortage, granted))


@_bindable("tq_pages_trim")
def tq_pages_trim(pool, table, lengths, window=0, sinks=0):
    """Gives back the pages that hold no token a query from position
    lengths[b] - 1 on sees."""
    a = tq_pages_trim_args(pool.struct(), _table_struct(table), _int32_ptr(lengths, "lengths", table.shape[0]),
                           _int_check(window, "window"), _int_check(sinks, "sinks"))
    _device_check(pool.refs, table=table, lengths=lengths)
    return BoundCall("tq_pages_trim", a, None, (pool, table, lengths))


@_bindable("tq_pages_fork")
def tq_pages_fork(pool, src, dst, parent, src_lengths, dst_lengths, workspace, keep_src=True, shortage=None):
    """Rows of dst become children of the rows parent[i] of src: full pages
    shared, a half-filled last page copied."""
    a = tq_pages_fork_args(pool.struct(), _table_struct(src), _table_struct(dst),
                           _int32_ptr(parent, "parent", dst.shape[0]),
                           _int32_ptr(src_lengths, "src_lengths", src.shape[0]),
                           _int32_ptr(dst_lengths, "dst_lengths", dst.shape[0]), 1 if keep_src else 0,
                           _int32_ptr(shortage, "shortage", 1))
    _device_check(pool.refs, src=src, dst=dst, parent=parent, src_lengths=src_lengths, dst_lengths=dst_lengths,
                  shortage=shortage, workspace=workspace)
    return BoundCall("tq_pages_fork", a, workspace,
                     (pool, src, dst, parent, src_lengths, dst_lengths, shortage))


@_bindable("tq_pages_copy")
def tq_pages_copy(src_pool, dst_pool, src_pages, dst_pages):
    """Copies page src_pages[i] of one pool into page dst_pages[i] of the other (or the same)."""
    n = src_pages.numel()
    a = tq_pages_copy_args(src_pool.struct(), dst_pool.struct(), _int32_ptr(src_pages, "src_pages"),
                           _int32_ptr(dst_pages, "dst_pages", n), n)
    _device_check(src_pool.refs, dst_pool=dst_pool.refs, src_pages=src_pages, dst_pages=dst_pages)
    return BoundCall("tq_pages_copy", a, None, (src_pool, dst_pool, src_pages, dst_pages))


@_bindable("tq_pages_compact")
def tq_pages_compact(src_pool, src_tables, dst_pool, dst_tables, workspace, live=None):
    """Moves the live pages to the lowest numbers: in place (the same pool and
    tables twice) or into another pool; a page table or a list of up to 4."""
    st = [src_tables] if hasattr(src_tables, "data_ptr") else list(src_tables)
    dt = [dst_tables] if hasattr(dst_tables, "data_ptr") else list(dst_tables)
    if len(st) != len(dt) or len(st) > TQ_MAX_PAGE_TABLES:
        raise ValueError("src_tables and dst_tables must be as many, at most 4")
    a = tq_pages_compact_args()
    a.src, a.dst = src_pool.struct(), dst_pool.struct()
    for i, (x, y) in enumerate(zip(st, dt)):
        a.src_tables[i], a.dst_tables[i] = _table_struct(x), _table_struct(y)
    a.n_tables = len(st)
    a.live = _int32_ptr(live, "live", 1)
    _device_check(src_pool.refs, dst_pool=dst_pool.refs, live=live, workspace=workspace,
                  **{f"table {i}": t for i, t in enumerate(st + dt)})
    return BoundCall("tq_pages_compact", a, workspace, (src_pool, st, dst_pool, dt, live))


TQ_DEVERR_SCAN_WAIT = 1
TQ_DEVERR_SELFTEST_WAIT = 2
TQ_DEVERR_QUANT_WAIT = 4
TQ_DEVERR_PAGE_WAIT = 8


def tq_device_errors(reset=False):
    """(status, flags) of the current device's error word; synchronises the device."""
    v = ctypes.c_uint32(0)
    st = load().tq_device_errors(ctypes.byref(v), 1 if reset else 0)
    if st not in (TQ_OK, TQ_ERR_TIMEOUT):
        _check(st, "tq_device_errors")
    return st, v.value


def tq_selftest_bounded_wait(limit_us, stream=None):
    """One warp waits on an mbarrier nothing arrives on, at most limit_us."""
    _check(load().tq_selftest_bounded_wait(limit_us, _stream_ptr(stream)), "tq_selftest_bounded_wait")


def tq_selftest_umma_gemm(a, b, d, stream=None, a_in_tmem=False):
    """d[128][n] = a[128][k] @ b[n][k]^T on the tcgen05 tensor-core path (fp16 in, fp32 out);
    a_in_tmem: the MMA reads A from tensor memory instead of shared memory."""
    n, k = b.shape
    fn = load().tq_selftest_umma_gemm_tmem_a if a_in_tmem else load().tq_selftest_umma_gemm
    _check(fn(a.data_ptr(), b.data_ptr(), d.data_ptr(), n, k, _stream_ptr(stream)), "tq_selftest_umma_gemm")


def _topk_struct(queries, db, n_db, rot, qjl, k, ids, scores):
    a = tq_topk_args()
    a.queries = queries.data_ptr()
    a.nq, a.d = queries.shape
    a.rot = rot.handle
    a.qjl = qjl.handle if qjl is not None else None
    a.db = db.struct()
    a.n_db = n_db
    a.k = k
    a.ids = ids.data_ptr()
    a.scores = scores.data_ptr()
    return a


def tq_score_topk_workspace(queries, db, n_db, rot, qjl, k, ids, scores):
    a = _topk_struct(queries, db, n_db, rot, qjl, k, ids, scores)
    return load().tq_score_topk_workspace(ctypes.byref(a))


def tq_score_topk(queries, db, n_db, rot, qjl, k, ids, scores, workspace, stream=None):
    a = _topk_struct(queries, db, n_db, rot, qjl, k, ids, scores)
    _check(load().tq_score_topk(ctypes.byref(a), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream_ptr(stream)), "tq_score_topk")


def workspace(nbytes, device="cuda"):
    """A 256-byte aligned device byte buffer (torch allocations are)."""
    import torch

    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class QuantizedKVCache:
    """One attention layer's packed KV cache with the decode loop's calls:
    `prefill` quantizes a context into it, `prefill_chunk` appends a chunk of
    tokens per batch row and attends with the chunk's queries (causal), and
    `step` appends one token per batch row and attends (the write-ups'
    "quantize on every cache update, then attend"; tq_quantize_kv,
    tq_attn_prefill and tq_decode_step). Keys are PROD (k_bits,
    QJL signs), values MSE (v_bits); both share one rotation. The per-row
    lengths live on the device; this class only keeps the handles, the
    planes and a workspace, and forms the calls' arguments."""

    def __init__(self, batch, hq, hkv, capacity, d=128, k_bits=3, v_bits=3, rotation="rht", rot_seed=1, qjl_seed=2,
                 device="cuda", k_bits2=None, v_bits2=None):
        import torch

        if hq % hkv:
            raise ValueError("hq must be a multiple of hkv")
        self.batch, self.hq, self.hkv, self.capacity, self.d = batch, hq, hkv, capacity, d
        self.rot = tq_rotation_to_device(tq_make_rotation(rot_seed, d, rotation))
        self.qjl = tq_qjl_to_device(tq_make_qjl(qjl_seed, d, d))
        self.k = Cache("prod", k_bits, d, rows=batch * hkv, capacity=capacity, device=device, bits2=k_bits2)
        self.v = Cache("mse", v_bits, d, rows=batch * hkv, capacity=capacity, device=device, bits2=v_bits2)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=device)
        self._host_lengths = [0] * batch  # the same lengths, for the launch plans
        self._ws = None

    def prefill(self, k, v, lengths):
        """k, v: device [batch, hkv, T, d] (f32 or bf16), T <= capacity; row b
        holds lengths[b] valid tokens (a host sequence of ints)."""
        import torch

        b, h, t, d = k.shape
        if (b, h, d) != (self.batch, self.hkv, self.d) or tuple(v.shape) != tuple(k.shape) or t > self.capacity:
            raise ValueError("k and v must be [batch, hkv, T <= capacity, d]")
        lens = [int(x) for x in lengths]
        if len(lens) != b or min(lens) < 0 or max(lens) > t:
            raise ValueError("lengths must give 0 <= length <= T per batch row")
        # slot of token j of (b, h): (b * hkv + h) * capacity + j; tokens past a row's length are skipped
        j = torch.arange(t, device=k.device, dtype=torch.int64)
        rows = torch.arange(b * h, device=k.device, dtype=torch.int64)
        slots = rows[:, None] * self.capacity + j[None, :]
        valid = j[None, :] < torch.tensor(lens, device=k.device, dtype=torch.int64).repeat_interleave(h)[:, None]
        slots = torch.where(valid, slots, torch.full_like(slots, -1)).reshape(-1).contiguous()
        tq_quantize_kv(self.k, self.rot, k.reshape(-1, d), qjl=self.qjl, dst_slot=slots)
        tq_quantize_kv(self.v, self.rot, v.reshape(-1, d), dst_slot=slots)
        self.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        self._host_lengths = lens

    def prefill_chunk(self, q, k, v, out=None, stream=None):
        """Appends a chunk of C tokens to every batch row (k, v: device
        [batch, hkv, C, d]) at the row's current length, then attends with the
        chunk's queries (device [batch, C, hq, d]; query i sees the row's
        tokens up to and including chunk token i). Returns out
        ([batch, C, hq, d], fp32 unless given)."""
        import torch

        b, h, c, d = k.shape
        if (b, h, d) != (self.batch, self.hkv, self.d) or tuple(v.shape) != tuple(k.shape):
            raise ValueError("k and v must be [batch, hkv, C, d]")
        if tuple(q.shape) != (b, c, self.hq, d):
            raise ValueError("q must be [batch, C, hq, d]")
        max_context = max(self._host_lengths) + c
        if max_context > self.capacity:
            raise ValueError("the chunk does not fit the capacity")
        if out is None:
            out = torch.empty((b, c, self.hq, d), dtype=torch.float32, device=q.device)
        # slot of chunk token j of (b, h): (b * hkv + h) * capacity + lengths[b] + j
        j = torch.arange(c, device=k.device, dtype=torch.int64)
        rows = torch.arange(b * h, device=k.device, dtype=torch.int64)
        start = self.lengths.to(torch.int64).repeat_interleave(h)
        slots = (rows[:, None] * self.capacity + start[:, None] + j[None, :]).reshape(-1).contiguous()
        tq_quantize_kv(self.k, self.rot, k.reshape(-1, d), qjl=self.qjl, dst_slot=slots, stream=stream)
        tq_quantize_kv(self.v, self.rot, v.reshape(-1, d), dst_slot=slots, stream=stream)
        need = tq_attn_prefill_workspace(q, self.k, self.v, self.lengths, max_context, self.rot, self.qjl, out)
        if self._ws is None or self._ws.numel() < need:
            self._ws = workspace(need, device=q.device)
        tq_attn_prefill(q, self.k, self.v, self.lengths, max_context, self.rot, self.qjl, out, self._ws,
                        stream=stream)
        self.lengths = self.lengths + c
        self._host_lengths = [x + c for x in self._host_lengths]
        return out

    def step(self, q, k_new, v_new, out=None, stream=None):
        """Appends k_new / v_new (device [batch, hkv, d]) at each row's current
        length and attends with q (device [batch, hq, d]); returns out
        ([batch, hq, d], fp32 unless given). The caller keeps every length
        below the capacity."""
        import torch

        if out is None:
            out = torch.empty((self.batch, self.hq, self.d), dtype=torch.float32, device=q.device)
        kn = k_new.reshape(self.batch * self.hkv, self.d)
        vn = v_new.reshape(self.batch * self.hkv, self.d)
        new_lens = self.lengths + 1
        need = tq_decode_step_workspace(q, self.k, self.v, new_lens, self.capacity, self.rot, self.qjl, out, kn, vn,
                                        self.lengths)
        if self._ws is None or self._ws.numel() < need:
            self._ws = workspace(need, device=q.device)
        tq_decode_step(q, self.k, self.v, new_lens, self.capacity, self.rot, self.qjl, out, kn, vn, self.lengths,
                       self._ws, stream=stream)
        self.lengths = new_lens
        self._host_lengths = [x + 1 for x in self._host_lengths]
        return out


class PagedKVCache:
    """One attention layer's packed KV cache in pages, with the calls of a
    generation loop: `prefill_chunk` and `step` reserve pages, append and
    attend (tq_pages_reserve, tq_quantize_kv, tq_attn_prefill_view,
    tq_decode_step_view) and, with a window, give back the pages it has passed
    (tq_pages_trim; a page goes once no later query sees it, nor one after a
    rollback of up to max_rollback tokens: the longest draft that a speculative
    decoder may take back); `fork` makes
    every row a child of some row, as beam search and sampling do
    (tq_pages_fork); `rollback` drops tokens or frees rows, `compact` moves the
    live pages together. Keys are PROD, values MSE. Lengths, tables and counts
    live on the device: no call waits for the GPU. `shortage` counts, on the
    device, the pages that calls asked for and did not get; a caller that sizes
    the pool for its rows never sees any. A token without a page is lost: its row
    does not grow by it, and goes on behind the tokens it has (`lengths`).

    All calls but `fork` may be captured in a graph (after one run outside, so
    that the workspace is there). How often it is replayed the object cannot
    know: from the first capture on, every call plans for max_tokens, tokens past
    it are dropped, and calls made outside afterwards need a `rollback` with
    at_most first."""

    def __init__(self, batch, hq, hkv, n_pages, max_tokens, page=64, d=128, k_bits=3, v_bits=3, window=0, sinks=0,
                 rotation="rht", rot_seed=1, qjl_seed=2, device="cuda", k_bits2=None, v_bits2=None, max_rollback=0):
        import torch

        if hq % hkv:
            raise ValueError("hq must be a multiple of hkv")
        if max_rollback < 0:
            raise ValueError("max_rollback must be >= 0")
        self.batch, self.hq, self.hkv, self.d, self.page = batch, hq, hkv, d, page
        self.max_rollback = max_rollback
        self.window, self.sinks = window, sinks
        self.max_pages = -(-max_tokens // page)
        self.max_tokens = self.max_pages * page
        self.rot = tq_rotation_to_device(tq_make_rotation(rot_seed, d, rotation))
        self.qjl = tq_qjl_to_device(tq_make_qjl(qjl_seed, d, d))
        self.k = Cache("prod", k_bits, d, rows=n_pages * hkv, capacity=page, device=device, bits2=k_bits2)
        self.v = Cache("mse", v_bits, d, rows=n_pages * hkv, capacity=page, device=device, bits2=v_bits2)
        self.pool = PagePool(self.k, self.v, hkv)
        self.table = self.pool.table(batch, self.max_pages)
        self._spare = self.pool.table(batch, self.max_pages)  # where a fork forms its rows; what it held is not counted
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=device)
        self.shortage = torch.zeros(1, dtype=torch.int32, device=device)
        self._short = torch.zeros(1, dtype=torch.int32, device=device)
        self._granted = torch.zeros(batch, dtype=torch.int32, device=device)  # tokens of the call that have a page
        self._bound = 0  # no row is longer, but for replays
        self._replays = False  # a call that appends was captured
        self._pages_ws = workspace(tq_pages_workspace(self.pool, batch), device=device)
        self._ws = None
        self._captured = []  # workspaces that graphs hold the addresses of

    def _view(self):
        return View(self.window, self.sinks, self.table, self.pool.n_pages)

    @staticmethod
    def _capturing(stream):
        import torch

        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            return torch.cuda.is_current_stream_capturing()

    def _reserve(self, add, stream):
        import torch

        if self._capturing(stream):
            self._bound, self._replays = self.max_tokens, True
        elif self._bound + add > self.max_tokens:
            raise ValueError("the tokens do not fit max_tokens (after replays, rollback's at_most says what is there)")
        tq_pages_reserve(self.pool, self.table, self.lengths, add, self._pages_ws, shortage=self._short,
                         granted=self._granted, stream=stream)
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            self.shortage += self._short

    def _inputs_check(self, q, k, v, out):
        """Before anything is enqueued; strided inputs are copied."""
        import torch

        for t, what in ((q, "q"), (k, "the keys"), (v, "the values")):
            if t.dtype not in (torch.float32, torch.bfloat16):
                raise ValueError(f"{what} must be float32 or bfloat16")
        if k.dtype != v.dtype:
            raise ValueError("keys and values must have the same dtype")
        if out is not None:
            _dense_check(out, "out", q.numel())
        _device_check(self.lengths, q=q, k=k, v=v, out=out)

    def _longest(self, add):
        """No row is longer with `add` more tokens."""
        return self.max_tokens if self._replays else min(self._bound + add, self.max_tokens)

    def _advance(self, add, stream):
        import torch

        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            self.lengths += self._granted
        self._bound = min(self._bound + add, self.max_tokens)
        if self.window > 0:
            self._trim(stream)

    def _trim(self, stream):
        """Gives back the pages that no query sees, now or after a rollback."""
        window = min(self.window + self.max_rollback, 2**31 - 1) if self.window > 0 else 0
        tq_pages_trim(self.pool, self.table, self.lengths, window, self.sinks, stream=stream)

    def _workspace(self, need, stream):
        import torch

        if self._ws is None or self._ws.numel() < need:
            with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
                if self._ws is not None:
                    # queued work may still use the one that goes, on another stream than its own
                    if torch.cuda.is_current_stream_capturing():
                        self._captured.append(self._ws)
                    else:
                        self._ws.record_stream(torch.cuda.current_stream())
                self._ws = workspace(need, device=self.lengths.device)
        if self._capturing(stream) and not any(w is self._ws for w in self._captured):
            self._captured.append(self._ws)
        return self._ws

    def prefill_chunk(self, q, k, v, out=None, stream=None):
        """Appends a chunk of C tokens to every row (k, v: device [batch, hkv,
        C, d]) and attends with its queries (device [batch, C, hq, d]);
        returns out ([batch, C, hq, d], fp32 unless given)."""
        import torch

        b, h, c, d = k.shape
        if (b, h, d) != (self.batch, self.hkv, self.d) or tuple(v.shape) != tuple(k.shape):
            raise ValueError("k and v must be [batch, hkv, C, d]")
        if tuple(q.shape) != (b, c, self.hq, d):
            raise ValueError("q must be [batch, C, hq, d]")
        self._inputs_check(q, k, v, out)
        self._reserve(c, stream)
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            if out is None:
                out = torch.empty((b, c, self.hq, d), dtype=torch.float32, device=q.device)
            q = q.contiguous()
            i = torch.arange(c, device=k.device)
            t = self.lengths.long()[:, None] + i
            e = self.table.long().gather(1, (t // self.page).clamp(max=self.max_pages - 1))[:, None, :]
            heads = torch.arange(h, device=k.device)[None, :, None]
            slots = torch.where((i < self._granted[:, None])[:, None, :],
                                (e * h + heads) * self.page + (t % self.page)[:, None, :], -1).reshape(-1)
            kr, vr = (x if x.stride(1) == 1 else x.contiguous() for x in (k.reshape(-1, d), v.reshape(-1, d)))
        tq_quantize_kv(self.k, self.rot, kr, qjl=self.qjl, dst_slot=slots, stream=stream)
        tq_quantize_kv(self.v, self.rot, vr, dst_slot=slots, stream=stream)
        a = (q, self.k, self.v, self.lengths, self._longest(c), self.rot, self.qjl, out)
        view = self._view()
        ws = self._workspace(tq_attn_prefill_view_workspace(*a, view), stream)
        tq_attn_prefill_view(*a, ws, view, stream=stream)
        self._advance(c, stream)
        return out

    def step(self, q, k_new, v_new, out=None, stream=None):
        """Appends k_new / v_new (device [batch, hkv, d]) to every row and
        attends with q (device [batch, hq, d]); returns out ([batch, hq, d],
        fp32 unless given)."""
        import torch

        if tuple(q.shape) != (self.batch, self.hq, self.d):
            raise ValueError("q must be [batch, hq, d]")
        n = self.batch * self.hkv * self.d
        if k_new.shape[-1:] != v_new.shape[-1:] or k_new.numel() != n or v_new.numel() != n:
            raise ValueError("k_new and v_new must be [batch, hkv, d]")
        self._inputs_check(q, k_new, v_new, out)
        self._reserve(1, stream)
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            if out is None:
                out = torch.empty((self.batch, self.hq, self.d), dtype=torch.float32, device=q.device)
            q, kn, vn = q.contiguous(), k_new.contiguous(), v_new.contiguous()  # the calls know no strides
            new_lens = self.lengths + self._granted
        a = (q, self.k, self.v, new_lens, self._longest(1), self.rot, self.qjl, out, kn, vn,
             self.lengths)
        view = self._view()
        ws = self._workspace(tq_decode_step_view_workspace(*a, view), stream)
        tq_decode_step_view(*a, ws, view, stream=stream)
        self._advance(1, stream)
        return out

    def _cut_lost(self, table, lengths):
        """Rows whose half-filled last page holds nothing end where it starts."""
        at = (lengths // self.page).clamp(max=self.max_pages - 1).long()
        lengths -= (lengths % self.page) * (table.gather(1, at[:, None])[:, 0] < 0)

    def fork(self, parent, stream=None):
        """Row i goes on from row parent[i] (device int32 [batch]; outside [0,
        batch): an empty row). Rows without a child are freed. The table and the
        lengths stay where they are, so that graphs captured before go on from
        them. Not captured itself (tq_pages_fork on a caller's own tables can be)."""
        import torch

        if self._capturing(stream):
            raise ValueError("PagedKVCache.fork cannot be captured")
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            lengths = torch.empty_like(self.lengths)
        tq_pages_fork(self.pool, self.table, self._spare, parent, self.lengths, lengths, self._pages_ws,
                      keep_src=False, shortage=self._short, stream=stream)
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            self.shortage += self._short
            self._cut_lost(self._spare, lengths)  # children that found no page for their copy
            self.table.copy_(self._spare)
            self.lengths.copy_(lengths)

    def rollback(self, lengths, at_most=None, stream=None):
        """Drops the tokens behind the first lengths[b] of every row (device
        int32 [batch]; a row that is no longer keeps its length; 0 frees it).
        at_most (an int): and those behind the first at_most, which tells the
        host how long the rows are where it knows a lower bound than the tokens
        appended so far (the calls plan with it and refuse what would pass
        max_tokens). Rows may go back to less than they were forked with: the
        page they go on in is copied by the next call that appends. With a window,
        a row that goes back by more than max_rollback tokens may find pages of its
        window gone: they count as shortage, their tokens are not visible, and
        where the row's last page is among them it goes on from that page's start."""
        import torch

        _int32_ptr(lengths, "lengths", self.batch)
        _device_check(self.lengths, lengths=lengths)
        if at_most is not None:
            at_most = max(int(at_most), 0)
            if not self._capturing(stream):  # else nothing has run yet
                self._bound = min(self._bound, at_most)
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            new = torch.minimum(self.lengths, lengths.clamp(min=0, max=at_most))
            if self.window > 0:
                # the pages with tokens of the window or the sinks
                j = torch.arange(self.max_pages, device=new.device)[None] * self.page
                n = new[:, None]
                seen = (j < n) & ((j + self.page > n - self.window) | (j < self.sinks))
                gone = seen & (self.table < 0) & (n < self.lengths[:, None])
                self.shortage += gone.sum().int()
                self._cut_lost(self.table, new)
            self.lengths.copy_(new)
        self._trim(stream)

    def compact(self, stream=None):
        """Moves the live pages to the lowest page numbers of the pool."""
        tq_pages_compact(self.pool, self.table, self.pool, self.table, self._pages_ws, stream=stream)
