"""Thin Python binding of the C-ABI library libtq.so (include/tq.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory (``tensor.data_ptr()``) and the
stream (``torch.cuda.current_stream().cuda_stream``).  Function names match
the C entry points.  There is no fallback: if libtq.so is missing, loading
raises.
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

TQ_OK = 0
STATUS = {0: "TQ_OK", 1: "TQ_ERR_INVALID_ARGUMENT", 2: "TQ_ERR_UNSUPPORTED",
          3: "TQ_ERR_CAPACITY", 4: "TQ_ERR_WORKSPACE", 5: "TQ_ERR_CUDA",
          6: "TQ_ERR_INTERNAL"}
TQ_F32, TQ_BF16, TQ_F16 = 0, 1, 2
TQ_VALUES_GROUP, TQ_VALUES_MSE = 0, 1
TILE_TOKENS = 128
MAX_BATCH = 1024

# Every function include/tq.h declares.
EXPORTS = ("tq_status_string", "tq_make_codebook", "tq_record_bytes", "tq_cache_bytes",
           "tq_quantize_append", "tq_decode_workspace_size", "tq_decode_attention",
           "tq_dequantize", "tq_decode_attention_noalloc", "tq_decode_attention_window",
           "tq_prefill_workspace_size", "tq_prefill_attention", "tq_prefill_tokens_per_pass",
           "tq_set_wait_limit_ns", "tq_device_errors", "tq_test_withhold_handoffs",
           "tq_test_sign_refine_threshold", "tq_test_refine_count", "tq_sketch_product", "tq_prepare_operands",
           "tq_make_rope_table", "tq_paged_bytes", "tq_paged_append", "tq_paged_gather", "tq_paged_decode_workspace_size",
           "tq_paged_decode_attention", "tq_prompt_attention")
ERRF_DECODE_WAIT, ERRF_QUANTIZE_WAIT, ERRF_PAGE, ERRF_POSITION, ERRF_PROMPT_WAIT = 1, 2, 4, 8, 16
NOALLOC_SCRATCH_BYTES = 8 << 20


class TQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


class Params(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("key_bits", ctypes.c_int),
                ("value_bits", ctypes.c_int), ("group", ctypes.c_int),
                ("pi", ctypes.c_void_p), ("s", ctypes.c_void_p),
                ("centroids", ctypes.c_void_p), ("boundaries", ctypes.c_void_p),
                ("value_mode", ctypes.c_int), ("v_centroids", ctypes.c_void_p),
                ("v_boundaries", ctypes.c_void_p), ("s_pit", ctypes.c_void_p),
                ("tc_operands", ctypes.c_void_p)]

TQ_TC_OPERAND_BYTES = 5 * 128 * 128 * 2


class Cache(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("h_kv", ctypes.c_int),
                ("capacity", ctypes.c_int), ("data", ctypes.c_void_p)]


class _PagedCacheStruct(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("h_kv", ctypes.c_int), ("page_tokens", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("data", ctypes.c_void_p)]


class _PagedBatchStruct(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("max_pages", ctypes.c_int), ("table_stride", ctypes.c_int),
                ("len", ctypes.c_void_p), ("block_table", ctypes.c_void_p)]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("max_positions", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("table", ctypes.c_void_p)]


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libtq.so (once) and declare its prototypes."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} not built; run python -m kv_cache_quantization_turboquantprod_b200.build")
    lib = ctypes.CDLL(p)
    P, C = ctypes.POINTER(Params), ctypes.POINTER(Cache)
    i32p = ctypes.POINTER(ctypes.c_int32)
    vp, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.tq_status_string.restype = ctypes.c_char_p
    lib.tq_status_string.argtypes = [ci]
    lib.tq_make_codebook.restype = ci
    lib.tq_make_codebook.argtypes = [ci, ci, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_double)]
    lib.tq_record_bytes.restype = sz
    lib.tq_record_bytes.argtypes = [P]
    lib.tq_sketch_product.restype = ci
    lib.tq_sketch_product.argtypes = [P, vp, vp]
    lib.tq_prepare_operands.restype = ci
    lib.tq_prepare_operands.argtypes = [P, vp, vp]
    lib.tq_cache_bytes.restype = sz
    lib.tq_cache_bytes.argtypes = [P, ci, ci, ci]
    lib.tq_quantize_append.restype = ci
    lib.tq_quantize_append.argtypes = [P, C, vp, vp, ci, ci, i32p, i32p, vp]
    lib.tq_decode_workspace_size.restype = sz
    lib.tq_decode_workspace_size.argtypes = [P, C, ci, ci]
    lib.tq_decode_attention.restype = ci
    lib.tq_decode_attention.argtypes = [P, C, vp, ci, ci, vp, ci, ctypes.c_float, vp, vp, sz, vp]
    lib.tq_decode_attention_noalloc.restype = ci
    lib.tq_decode_attention_noalloc.argtypes = [P, C, vp, ci, ci, vp, ci, ctypes.c_float, vp, vp]
    lib.tq_decode_attention_window.restype = ci
    lib.tq_decode_attention_window.argtypes = [P, C, vp, ci, ci, vp, ci, vp, vp, ci, vp, ci,
                                               ctypes.c_float, vp, vp, sz, vp]
    lib.tq_prefill_workspace_size.restype = sz
    lib.tq_prefill_workspace_size.argtypes = [P, C, ci, ci, ci]
    lib.tq_prefill_tokens_per_pass.restype = ci
    lib.tq_prefill_tokens_per_pass.argtypes = [P, ci, ci, ci]
    lib.tq_prefill_attention.restype = ci
    lib.tq_prefill_attention.argtypes = [P, C, vp, ci, ci, ci, vp, ci, ctypes.c_float, vp, vp, sz, vp]
    lib.tq_dequantize.restype = ci
    lib.tq_dequantize.argtypes = [P, C, ci, ci, ci, vp, vp, vp]
    cll = ctypes.c_longlong
    PC, PB, PR = (ctypes.POINTER(t) for t in (_PagedCacheStruct, _PagedBatchStruct, _RopeStruct))
    lib.tq_make_rope_table.restype = ci
    lib.tq_make_rope_table.argtypes = [ci, ci, ctypes.c_double, vp]
    lib.tq_paged_bytes.restype = sz
    lib.tq_paged_bytes.argtypes = [ci, ci, ci, ci]
    lib.tq_paged_append.restype = ci
    lib.tq_paged_append.argtypes = [PC, PB, PR, vp, vp, vp, vp, ci, ci, ci, cll, cll, cll, vp, vp, cll, cll, vp]
    lib.tq_paged_gather.restype = ci
    lib.tq_paged_gather.argtypes = [PC, PB, vp, vp, ci, vp, vp, ci, cll, cll, vp]
    lib.tq_paged_decode_workspace_size.restype = sz
    lib.tq_paged_decode_workspace_size.argtypes = [PC, ci, ci]
    lib.tq_paged_decode_attention.restype = ci
    lib.tq_paged_decode_attention.argtypes = [PC, PB, vp, ci, ci, cll, ctypes.c_float, vp, cll, vp, sz, vp]
    lib.tq_prompt_attention.restype = ci
    lib.tq_prompt_attention.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci, ci, cll, cll, cll, vp, vp, ci,
                                        ctypes.c_float, vp, cll, vp]
    lib.tq_set_wait_limit_ns.restype = ci
    lib.tq_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.tq_test_withhold_handoffs.restype = ci
    lib.tq_test_withhold_handoffs.argtypes = [ci]
    lib.tq_test_sign_refine_threshold.restype = ci
    lib.tq_test_sign_refine_threshold.argtypes = [ctypes.c_double]
    lib.tq_test_refine_count.restype = ci
    lib.tq_test_refine_count.argtypes = [ctypes.POINTER(ctypes.c_ulonglong), ci]
    lib.tq_device_errors.restype = ci
    lib.tq_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32), ci]
    if path is None:
        _lib = lib
    return lib


def _check(fn: str, st: int) -> None:
    if st != TQ_OK:
        raise TQError(fn, st)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TQ_F32
    if t.dtype == torch.bfloat16:
        return TQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check_rows(name: str, t: torch.Tensor, shape, dtypes, device=None) -> None:
    """Shape, dtype, contiguity and device of a tensor handed to the C ABI,
    which cannot check buffer sizes itself."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor on the cache's device")


def _check_decode_io(cache, q: torch.Tensor, len_dev: torch.Tensor, out: torch.Tensor) -> int:
    """q [B, H_q, d] fp32/bf16, len_dev [B] int32, out [B, H_q, d] fp32, all
    contiguous on the cache's device; returns H_q."""
    if q.dim() != 3:
        raise ValueError("q must be [B, H_q, d]")
    dev = cache.buffer.device
    B, hq, d = cache.batch, int(q.shape[1]), int(q.shape[2])
    _check_rows("q", q, (B, hq, d), (torch.float32, torch.bfloat16), dev)
    _check_rows("len_dev", len_dev, (B,), (torch.int32,), dev)
    _check_rows("out", out, (B, hq, d), (torch.float32,), dev)
    return hq


def _i32_array(xs):
    arr = (ctypes.c_int32 * len(xs))(*[int(x) for x in xs])
    return arr


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def tq_status_string(status: int) -> str:
    return load().tq_status_string(int(status)).decode()


def tq_make_codebook(mse_bits: int, d: int):
    """Host-only Lloyd-Max codebook: (centroids [2^b], boundaries [2^b - 1]) as
    Python float lists."""
    n = 1 << mse_bits if 1 <= mse_bits <= 4 else 1
    c = (ctypes.c_double * n)()
    b = (ctypes.c_double * max(n - 1, 1))()
    _check("tq_make_codebook", load().tq_make_codebook(mse_bits, d, c, b))
    return list(c), list(b)[: n - 1]


class Layer:
    """Device-resident constants of one layer (Pi, S, codebooks) packaged as
    the C struct tq_params.  Holds references to the tensors it points to.
    value_mode "group" (min/max groups of 32) or "mse" (TurboQuant-MSE values
    with the value_bits Lloyd-Max codebook)."""

    def __init__(self, pi, s, key_bits: int, value_bits: int, group: int = 32,
                 device="cuda", value_mode: str = "group"):
        d = int(pi.shape[0])
        cent, bnd = tq_make_codebook(key_bits - 1, d)
        self.pi = torch.as_tensor(pi, dtype=torch.float32).contiguous().to(device)
        self.s = torch.as_tensor(s, dtype=torch.float32).contiguous().to(device)
        self.centroids = torch.tensor(cent, dtype=torch.float32, device=device)
        self.boundaries = torch.tensor(bnd if bnd else [0.0], dtype=torch.float32, device=device)
        self.codebook = (cent, bnd)
        self.value_mode = value_mode
        mode = {"group": TQ_VALUES_GROUP, "mse": TQ_VALUES_MSE}[value_mode]
        vc_ptr = vb_ptr = None
        if mode == TQ_VALUES_MSE:
            vcent, vbnd = tq_make_codebook(value_bits, d)
            self.v_centroids = torch.tensor(vcent, dtype=torch.float32, device=device)
            self.v_boundaries = torch.tensor(vbnd, dtype=torch.float32, device=device)
            self.value_codebook = (vcent, vbnd)
            vc_ptr, vb_ptr = self.v_centroids.data_ptr(), self.v_boundaries.data_ptr()
        # W = S Pi^T in float64, for the append kernels' sign refinement and
        # sketch; at d = 128 also the tensor-core append's operand images
        self.s_pit = torch.empty((d, d), dtype=torch.float64, device=device)
        on_gpu = self.s_pit.is_cuda
        self.tc_operands = (torch.empty(TQ_TC_OPERAND_BYTES, dtype=torch.uint8, device=device)
                            if on_gpu and d == 128 else None)
        self.params = Params(d, key_bits, value_bits, group, self.pi.data_ptr(),
                             self.s.data_ptr(), self.centroids.data_ptr(),
                             self.boundaries.data_ptr(), mode, vc_ptr, vb_ptr,
                             self.s_pit.data_ptr(),
                             self.tc_operands.data_ptr() if self.tc_operands is not None else None)
        if on_gpu:
            tq_sketch_product(self)
            if self.tc_operands is not None:
                tq_prepare_operands(self)

    @property
    def d(self):
        return self.params.d

    def record_bytes(self) -> int:
        return int(load().tq_record_bytes(ctypes.byref(self.params)))


class CompressedCache:
    """A caller-owned cache buffer (torch uint8 tensor) as the C struct
    tq_cache."""

    def __init__(self, layer: Layer, batch: int, h_kv: int, capacity: int,
                 device="cuda", zero: bool = False):
        n = tq_cache_bytes(layer, batch, h_kv, capacity)
        if n == 0:
            raise TQError("tq_cache_bytes", 1)
        alloc = torch.zeros if zero else torch.empty
        self.buffer = alloc(n, dtype=torch.uint8, device=device)
        self.cache = Cache(batch, h_kv, capacity, self.buffer.data_ptr())
        self.batch, self.h_kv, self.capacity = batch, h_kv, capacity


def tq_sketch_product(layer: Layer, stream=None) -> None:
    """Write W = S Pi^T (float64) into layer.s_pit from the layer's Pi and S."""
    st = load().tq_sketch_product(ctypes.byref(layer.params), layer.s_pit.data_ptr(), _stream(stream))
    _check("tq_sketch_product", st)


def tq_prepare_operands(layer: Layer, stream=None) -> None:
    """Write the tensor-core append's operand images of the layer's Pi and
    W into layer.tc_operands (after tq_sketch_product)."""
    st = load().tq_prepare_operands(ctypes.byref(layer.params), layer.tc_operands.data_ptr(), _stream(stream))
    _check("tq_prepare_operands", st)


def tq_record_bytes(layer: Layer) -> int:
    return int(load().tq_record_bytes(ctypes.byref(layer.params)))


def tq_cache_bytes(layer: Layer, batch: int, h_kv: int, capacity: int) -> int:
    return int(load().tq_cache_bytes(ctypes.byref(layer.params), batch, h_kv, capacity))


def tq_quantize_append(layer: Layer, cache: CompressedCache, k: torch.Tensor,
                       v: torch.Tensor, len_host, n_new_host=None, stream=None) -> None:
    """k, v: [B, T, H_kv, d] device tensors (fp32 or bf16, contiguous)."""
    if k.dtype != v.dtype:
        raise TypeError("k and v must share a dtype")
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k and v must be contiguous")
    T = int(k.shape[1]) if k.dim() == 4 else 0
    lens = _i32_array(len_host)
    nn = _i32_array(n_new_host) if n_new_host is not None else None
    st = load().tq_quantize_append(ctypes.byref(layer.params), ctypes.byref(cache.cache),
                                   k.data_ptr(), v.data_ptr(), _dtype_code(k), T, lens,
                                   nn, _stream(stream))
    _check("tq_quantize_append", st)


def tq_decode_workspace_size(layer: Layer, cache: CompressedCache, h_q: int, max_len: int) -> int:
    return int(load().tq_decode_workspace_size(ctypes.byref(layer.params),
                                               ctypes.byref(cache.cache), h_q, max_len))


def tq_decode_attention(layer: Layer, cache: CompressedCache, q: torch.Tensor,
                        len_dev: torch.Tensor, max_len: int, out: torch.Tensor,
                        workspace: torch.Tensor, softmax_scale: float | None = None,
                        stream=None) -> None:
    """q [B, H_q, d] (fp32/bf16), len_dev [B] int32 device, out [B, H_q, d]
    fp32, workspace a uint8 device tensor."""
    hq = _check_decode_io(cache, q, len_dev, out)
    scale = (1.0 / layer.d ** 0.5) if softmax_scale is None else float(softmax_scale)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    st = load().tq_decode_attention(ctypes.byref(layer.params), ctypes.byref(cache.cache),
                                    q.data_ptr(), _dtype_code(q), hq,
                                    len_dev.data_ptr(), int(max_len), scale, out.data_ptr(),
                                    workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _check("tq_decode_attention", st)


def tq_decode_attention_window(layer: Layer, cache: CompressedCache, q: torch.Tensor,
                               len_dev: torch.Tensor, max_len: int, win_k: torch.Tensor,
                               win_v: torch.Tensor, win_len_dev: torch.Tensor, out: torch.Tensor,
                               workspace: torch.Tensor, softmax_scale: float | None = None,
                               stream=None) -> None:
    """Decode over the compressed cache plus a window of recent tokens kept
    exactly: win_k, win_v [B, H_kv, win_cap, d] (fp32/bf16, contiguous),
    win_len_dev [B] int32 device (valid slots per sequence)."""
    hq = _check_decode_io(cache, q, len_dev, out)
    if win_k.dim() != 4:
        raise ValueError("win_k must be [B, H_kv, win_cap, d]")
    wshape = (cache.batch, cache.h_kv, int(win_k.shape[2]), int(q.shape[2]))
    _check_rows("win_k", win_k, wshape, (torch.float32, torch.bfloat16), cache.buffer.device)
    _check_rows("win_v", win_v, wshape, (win_k.dtype,), cache.buffer.device)
    _check_rows("win_len_dev", win_len_dev, (cache.batch,), (torch.int32,), cache.buffer.device)
    scale = (1.0 / layer.d ** 0.5) if softmax_scale is None else float(softmax_scale)
    st = load().tq_decode_attention_window(ctypes.byref(layer.params), ctypes.byref(cache.cache),
                                           q.data_ptr(), _dtype_code(q), hq,
                                           len_dev.data_ptr(), int(max_len), win_k.data_ptr(),
                                           win_v.data_ptr(), _dtype_code(win_k), win_len_dev.data_ptr(),
                                           int(win_k.shape[2]), scale, out.data_ptr(),
                                           workspace.data_ptr(),
                                           workspace.numel() * workspace.element_size(),
                                           _stream(stream))
    _check("tq_decode_attention_window", st)


def tq_decode_attention_noalloc(layer: Layer, cache: CompressedCache, q: torch.Tensor,
                                len_dev: torch.Tensor, max_len: int, out: torch.Tensor,
                                softmax_scale: float | None = None, stream=None) -> None:
    """Decode attention for callers that cannot allocate a workspace: the
    scratch is the library's fixed 8 MiB device array (see include/tq.h)."""
    hq = _check_decode_io(cache, q, len_dev, out)
    scale = (1.0 / layer.d ** 0.5) if softmax_scale is None else float(softmax_scale)
    st = load().tq_decode_attention_noalloc(ctypes.byref(layer.params), ctypes.byref(cache.cache),
                                            q.data_ptr(), _dtype_code(q), hq,
                                            len_dev.data_ptr(), int(max_len), scale,
                                            out.data_ptr(), _stream(stream))
    _check("tq_decode_attention_noalloc", st)


def tq_prefill_workspace_size(layer: Layer, cache: CompressedCache, h_q: int, t_chunk: int,
                              max_len: int) -> int:
    return int(load().tq_prefill_workspace_size(ctypes.byref(layer.params), ctypes.byref(cache.cache),
                                                h_q, t_chunk, max_len))


def tq_prefill_attention(layer: Layer, cache: CompressedCache, q: torch.Tensor,
                         len_dev: torch.Tensor, max_len: int, out: torch.Tensor,
                         workspace: torch.Tensor, softmax_scale: float | None = None,
                         stream=None) -> None:
    """Causal attention of a chunk over the compressed cache (the chunk already
    appended): q [B, T, H_q, d] (fp32/bf16, contiguous), len_dev [B] int32
    device (cached tokens, the chunk included), out [B, T, H_q, d] fp32."""
    if q.dim() != 4:
        raise ValueError("q must be a contiguous [B, T, H_q, d] tensor")
    dev = cache.buffer.device
    _check_rows("q", q, (cache.batch,) + tuple(q.shape[1:]), (torch.float32, torch.bfloat16), dev)
    _check_rows("len_dev", len_dev, (cache.batch,), (torch.int32,), dev)
    _check_rows("out", out, tuple(q.shape), (torch.float32,), dev)
    scale = (1.0 / layer.d ** 0.5) if softmax_scale is None else float(softmax_scale)
    st = load().tq_prefill_attention(ctypes.byref(layer.params), ctypes.byref(cache.cache),
                                     q.data_ptr(), _dtype_code(q), int(q.shape[2]), int(q.shape[1]),
                                     len_dev.data_ptr(), int(max_len), scale, out.data_ptr(),
                                     workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     _stream(stream))
    _check("tq_prefill_attention", st)


def tq_prefill_tokens_per_pass(layer: Layer, h_q: int, h_kv: int, t_chunk: int) -> int:
    return int(load().tq_prefill_tokens_per_pass(ctypes.byref(layer.params), h_q, h_kv, t_chunk))


def prefill_workspace_for(layer: Layer, cache: CompressedCache, h_q: int, t_chunk: int,
                          max_len: int, device="cuda") -> torch.Tensor:
    n = tq_prefill_workspace_size(layer, cache, h_q, t_chunk, max_len)
    if n == 0:
        raise TQError("tq_prefill_workspace_size", 1)
    return torch.empty(n, dtype=torch.uint8, device=device)


def tq_set_wait_limit_ns(ns: int) -> None:
    """Time limit of the kernels' bounded waits for later calls (0: the
    default, 2 s).  For tests of the timeout path."""
    _check("tq_set_wait_limit_ns", load().tq_set_wait_limit_ns(int(ns)))


def tq_test_withhold_handoffs(on: bool | int) -> None:
    """Tests of the timeout path: make later calls' tensor-core kernels
    withhold one hand-off so that their bounded waits run out (2: see
    include/tq.h)."""
    _check("tq_test_withhold_handoffs", load().tq_test_withhold_handoffs(int(on)))


def tq_test_sign_refine_threshold(z: float) -> None:
    """Tests of the float64 sign refinement: later appends re-decide every
    QJL sign with |(S r)_j| < z in float64 (0: the default, 1e-5)."""
    _check("tq_test_sign_refine_threshold", load().tq_test_sign_refine_threshold(float(z)))


def tq_test_refine_count(clear: bool = False) -> int:
    """Synchronise the device; QJL sign bits re-decided in float64 by the
    append kernels since the last reset (reset it when ``clear``)."""
    n = ctypes.c_ulonglong(0)
    _check("tq_test_refine_count", load().tq_test_refine_count(ctypes.byref(n), int(bool(clear))))
    return int(n.value)


def tq_device_errors(clear: bool = False) -> int:
    """Synchronise the current device and return its sticky error word
    (ERRF_* bits of kernels that gave up on a bounded wait); optionally
    reset it."""
    v = ctypes.c_uint32(0)
    _check("tq_device_errors", load().tq_device_errors(ctypes.byref(v), int(bool(clear))))
    return int(v.value)


def decode_status(workspace: torch.Tensor) -> int:
    """The status word a decode call left in its workspace (first int32):
    nonzero if a kernel of that call gave up on a bounded wait."""
    return int(workspace[:4].view(torch.int32).item())


def tq_dequantize(layer: Layer, cache: CompressedCache, b: int, start: int, count: int,
                  k_out: torch.Tensor, v_out: torch.Tensor, stream=None) -> None:
    st = load().tq_dequantize(ctypes.byref(layer.params), ctypes.byref(cache.cache), b, start,
                              count, k_out.data_ptr(), v_out.data_ptr(), _stream(stream))
    _check("tq_dequantize", st)


def workspace_for(layer: Layer, cache: CompressedCache, h_q: int, max_len: int,
                  device="cuda") -> torch.Tensor:
    n = tq_decode_workspace_size(layer, cache, h_q, max_len)
    if n == 0:
        raise TQError("tq_decode_workspace_size", 1)
    return torch.empty(n, dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# paged 4-bit cache and prompt attention
# ---------------------------------------------------------------------------
_PAGED_DTYPES = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}
_HALF_DTYPES = {torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}


def _token_rows(name: str, t: torch.Tensor, heads: int, d: int, dtype, device, rows: int) -> int:
    """Check [rows, heads, d] token rows whose heads are contiguous (tokens may lie further apart); returns the tokens'
    stride in elements."""
    if t.shape != (rows, heads, d):
        raise ValueError(f"{name} must be [{rows}, {heads}, {d}], got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    stride, by_head, by_channel = t.stride()
    if by_channel != 1 or (by_head != d and heads > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous rows")
    return stride if rows > 1 else heads * d  # (one row's stride means nothing)


def _three_dims(name: str, t: torch.Tensor):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, d], got {tuple(t.shape)}")
    return t.shape


def _int32(name: str, t: torch.Tensor, n: int, device) -> int:
    if t.dtype is not torch.int32 or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [{n}] on {device}")
    return t.data_ptr()


def _call(fn, device, stream, *args) -> int:
    """fn(*args, stream handle) with `device` current: its kernels run there whatever device the caller has selected, on the
    device's current stream where none is given."""
    index = device.index
    if torch._C._cuda_getDevice() == index:
        return fn(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream))
    with torch.cuda.device(device):
        return fn(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream))


def tq_make_rope_table(max_positions: int, rotary_dim: int, theta: float = 10000.0) -> torch.Tensor:
    """Host table [max_positions, rotary_dim] float32: cosines, then sines, of the angles p theta^(-2 j / rotary_dim)."""
    table = torch.empty(max(int(max_positions), 1), max(int(rotary_dim), 1), dtype=torch.float32)
    _check("tq_make_rope_table", load().tq_make_rope_table(int(max_positions), int(rotary_dim), float(theta), table.data_ptr()))
    return table


def tq_paged_bytes(d: int, h_kv: int, page_tokens: int, num_pages: int) -> int:
    return int(load().tq_paged_bytes(d, h_kv, page_tokens, num_pages))


class PagedCache:
    """A pool of 4-bit pages (include/tq.h, tq_paged_cache) in a caller-owned uint8 tensor; allocated where none is given."""

    def __init__(self, d: int, h_kv: int, page_tokens: int, num_pages: int, buffer: torch.Tensor | None = None, device="cuda"):
        n = tq_paged_bytes(d, h_kv, page_tokens, num_pages)
        if n == 0:
            raise TQError("tq_paged_bytes", 1)
        if buffer is None:
            buffer = torch.empty(n, dtype=torch.uint8, device=device)
        if buffer.dtype != torch.uint8 or not buffer.is_contiguous() or buffer.numel() < n or not buffer.is_cuda:
            raise ValueError(f"buffer must be a contiguous CUDA uint8 tensor of at least {n} bytes")
        self.buffer, self.device = buffer, buffer.device
        self.d, self.h_kv, self.page_tokens, self.num_pages = d, h_kv, page_tokens, num_pages
        self.struct = _PagedCacheStruct(d, h_kv, page_tokens, num_pages, buffer.data_ptr())
        self.ref = ctypes.byref(self.struct)


class PagedBatch:
    """Lengths [B] int32 (the tokens that a call appends included) and block table [B, max_pages] int32 on the device.
    The tensors are read when a call's kernels run, so a loop updates them in place."""

    def __init__(self, len_dev: torch.Tensor, block_table: torch.Tensor):
        if len_dev.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] != len_dev.shape[0]:
            raise ValueError("len_dev must be [B] and block_table [B, max_pages]")
        if len_dev.dtype != torch.int32 or block_table.dtype != torch.int32:
            raise TypeError("len_dev and block_table must be int32")
        if not len_dev.is_cuda or block_table.device != len_dev.device:
            raise ValueError("len_dev and block_table must be CUDA tensors on one device")
        if not len_dev.is_contiguous() or (block_table.stride(1) != 1 and block_table.shape[1] > 1):
            raise ValueError("len_dev and the rows of block_table must be contiguous")
        self.len_dev, self.block_table, self.device = len_dev, block_table, len_dev.device
        self.batch, self.max_pages = (int(x) for x in block_table.shape)
        stride = int(block_table.stride(0)) if self.batch > 1 else self.max_pages
        self.struct = _PagedBatchStruct(self.batch, self.max_pages, stride, len_dev.data_ptr(), block_table.data_ptr())
        self.ref = ctypes.byref(self.struct)


class Rope:
    """A rotation table [max_positions, rotary_dim] float32 on the device (tq_make_rope_table's layout); ``interleaved``
    turns adjacent channels instead of the two halves."""

    def __init__(self, table: torch.Tensor, interleaved: bool = False):
        if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous() or not table.is_cuda:
            raise ValueError("table must be a contiguous CUDA float32 tensor [max_positions, rotary_dim]")
        self.table, self.device = table, table.device
        self.struct = _RopeStruct(int(table.shape[1]), int(table.shape[0]), int(bool(interleaved)), table.data_ptr())
        self.ref = ctypes.byref(self.struct)


def _same_device(cache: PagedCache, batch: PagedBatch) -> None:
    if batch.device != cache.device:
        raise ValueError(f"the batch's tensors must be on the cache's device {cache.device}, got {batch.device}")


def tq_paged_append(cache: PagedCache, batch: PagedBatch, cu_new: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    q: torch.Tensor | None = None, rope: Rope | None = None, q_out: torch.Tensor | None = None,
                    k_out: torch.Tensor | None = None, stream=None) -> None:
    """Rotate and store new tokens: k, v [T, H_kv, d] and optionally q [T, H_q, d] (fp32, bf16 or fp16; tokens may lie
    further apart than their rows), cu_new [B + 1] int32; rotated rows to q_out and k_out where given."""
    dev, d, dt = cache.device, cache.d, k.dtype
    _same_device(cache, batch)
    if dt not in _PAGED_DTYPES:
        raise TypeError(f"unsupported dtype {dt}")
    T = k.shape[0]
    ks = _token_rows("k", k, cache.h_kv, d, dt, dev, T)
    vs = _token_rows("v", v, cache.h_kv, d, dt, dev, T)
    kos, kp = (_token_rows("k_out", k_out, cache.h_kv, d, dt, dev, T), k_out.data_ptr()) if k_out is not None else (0, None)
    qs = qos = hq = 0
    qp = qop = None
    if q is not None:
        if q_out is None:
            raise ValueError("q needs q_out")
        hq = _three_dims("q", q)[1]
        qs = _token_rows("q", q, hq, d, dt, dev, T)
        qos = _token_rows("q_out", q_out, hq, d, dt, dev, T)
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if rope is not None and rope.device != dev:
        raise ValueError(f"the rotation table must be on {dev}, got {rope.device}")
    cu = _int32("cu_new", cu_new, batch.batch + 1, dev)
    st = _call(load().tq_paged_append, dev, stream, cache.ref, batch.ref, rope.ref if rope is not None else None, cu, qp,
               k.data_ptr(), v.data_ptr(), _PAGED_DTYPES[dt], hq, T, qs, ks, vs, qop, kp, qos, kos)
    _check("tq_paged_append", st)


def tq_paged_gather(cache: PagedCache, batch: PagedBatch, cu_rows: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor,
                    first: torch.Tensor | None = None, stream=None) -> None:
    """Cached tokens as rows of k_out, v_out [rows, H_kv, d] (fp32, bf16 or fp16): rows cu_rows[b] .. cu_rows[b + 1] - 1
    get sequence b's tokens from position first[b] (0 where first is None)."""
    dev, d, dt = cache.device, cache.d, k_out.dtype
    _same_device(cache, batch)
    if dt not in _PAGED_DTYPES:
        raise TypeError(f"unsupported dtype {dt}")
    rows = k_out.shape[0]
    ks = _token_rows("k_out", k_out, cache.h_kv, d, dt, dev, rows)
    vs = _token_rows("v_out", v_out, cache.h_kv, d, dt, dev, rows)
    cu = _int32("cu_rows", cu_rows, batch.batch + 1, dev)
    at = _int32("first", first, batch.batch, dev) if first is not None else None
    st = _call(load().tq_paged_gather, dev, stream, cache.ref, batch.ref, cu, at, rows, k_out.data_ptr(), v_out.data_ptr(),
               _PAGED_DTYPES[dt], ks, vs)
    _check("tq_paged_gather", st)


def tq_paged_decode_workspace_size(cache: PagedCache, batch: int, h_q: int) -> int:
    with torch.cuda.device(cache.device):
        return int(load().tq_paged_decode_workspace_size(cache.ref, batch, h_q))


def paged_workspace_for(cache: PagedCache, batch: PagedBatch, h_q: int) -> torch.Tensor:
    n = tq_paged_decode_workspace_size(cache, batch.batch, h_q)
    if n == 0:
        raise TQError("tq_paged_decode_workspace_size", 1)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def tq_paged_decode_attention(cache: PagedCache, batch: PagedBatch, q: torch.Tensor, out: torch.Tensor,
                              workspace: torch.Tensor, softmax_scale: float | None = None, stream=None) -> None:
    """Decode attention over the paged 4-bit cache: q, out [B, H_q, d] (bf16 or fp16), workspace a uint8 device tensor
    (paged_workspace_for) that no other call in flight uses."""
    dev, d, dt = cache.device, cache.d, q.dtype
    _same_device(cache, batch)
    if dt not in _HALF_DTYPES:
        raise TypeError(f"unsupported dtype {dt}")
    hq = _three_dims("q", q)[1]
    qs = _token_rows("q", q, hq, d, dt, dev, batch.batch)
    os_ = _token_rows("out", out, hq, d, dt, dev, batch.batch)
    if workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    scale = (1.0 / d ** 0.5) if softmax_scale is None else float(softmax_scale)
    st = _call(load().tq_paged_decode_attention, dev, stream, cache.ref, batch.ref, q.data_ptr(), _HALF_DTYPES[dt], hq, qs,
               scale, out.data_ptr(), os_, workspace.data_ptr(), workspace.numel())
    _check("tq_paged_decode_attention", st)


def tq_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                        out: torch.Tensor, softmax_scale: float | None = None, stream=None) -> None:
    """Causal attention of packed sequences: q, out [T_q, H_q, d], k, v [T_k, H_kv, d] (bf16 or fp16; tokens may lie
    further apart than their rows), cu_q, cu_k [B + 1] int32.  Query i of a sequence sees keys j <= i + n_k - n_q."""
    dev, dt = q.device, q.dtype
    if dt not in _HALF_DTYPES:
        raise TypeError(f"unsupported dtype {dt}")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    Tq, hq, d = _three_dims("q", q)
    Tk, hkv, _ = _three_dims("k", k)
    qs = _token_rows("q", q, hq, d, dt, dev, Tq)
    os_ = _token_rows("out", out, hq, d, dt, dev, Tq)
    ks = _token_rows("k", k, hkv, d, dt, dev, Tk)
    vs = _token_rows("v", v, hkv, d, dt, dev, Tk)
    if cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise ValueError("cu_q must be [B + 1] with B >= 1")
    B = cu_q.shape[0] - 1
    scale = (1.0 / d ** 0.5) if softmax_scale is None else float(softmax_scale)
    st = _call(load().tq_prompt_attention, dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), _HALF_DTYPES[dt], Tq, Tk, hq,
               hkv, d, qs, ks, vs, _int32("cu_q", cu_q, B + 1, dev), _int32("cu_k", cu_k, B + 1, dev), B, scale, out.data_ptr(),
               os_)
    _check("tq_prompt_attention", st)
