"""ctypes binding of libhisparse.so, the C ABI declared in include/hisparse.h.

Argument marshalling only: every computation runs in the library's CUDA
kernels. Tensors are passed by ``data_ptr()`` and the stream is torch's current
stream unless one is given. Importing this module loads the library and raises
ImportError when it has not been built, so nothing can silently fall back.
"""
from __future__ import annotations

import ctypes
import os
import struct
import sys
from array import array
from typing import Optional, Sequence

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhisparse.so")

STATUS = {
    0: "HS_OK", 1: "HS_ERR_INVALID", 2: "HS_ERR_OOM", 3: "HS_ERR_CAPACITY", 4: "HS_ERR_CUDA",
    5: "HS_ERR_TIMEOUT", 6: "HS_ERR_HOST_MISSING", 7: "HS_ERR_BAD_ID", 8: "HS_ERR_BAD_WEIGHT",
    9: "HS_ERR_SCRATCH_LIMIT", 10: "HS_ERR_NOT_RESOLVED", 11: "HS_ERR_RANGE",
}
SELECT_AUTO, SELECT_LOCAL = 0, 1   # HS_SELECT_AUTO, HS_SELECT_LOCAL
PLAN_PAD, PLAN_RESIDENT, PLAN_HIT, PLAN_MISS = 0, 1, 2, 3
IDX_INT8, IDX_FP8 = 0, 1       # HS_IDX_INT8, HS_IDX_FP8
IDX_FP8_PAGE_BYTES = 8448      # 64 x 128 e4m3 key bytes, then 64 fp32 scales
MAX_CTX = 1310720            # HS_MAX_CTX: longest context a pool accepts


class HisparseError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call}: {STATUS.get(status, status)}")
        self.status = status


class PoolConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "page_size", "row_bytes", "idx_dim", "n_idx_heads", "n_heads", "topk", "n_layers",
        "layers_per_indexer", "num_pages", "num_idx_pages", "max_requests", "max_ctx",
        "max_q_per_req", "hot_rows", "max_tokens", "idx_format")] + [("host_pages", ctypes.c_int64)]


class PlanEntry(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("slot", ctypes.c_int32), ("row", ctypes.c_int32),
                ("evicted", ctypes.c_int32)]


class Counters(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("resident", "hits", "misses", "h2d_bytes", "d2h_bytes")] + \
               [("reserved", ctypes.c_uint64 * 3)]


BF16, FP16, FP32 = 0, 1, 2   # HS_BF16, HS_FP16, HS_FP32
CACHE_MAX_TOKENS = 1 << 24   # HS_CACHE_MAX_TOKENS
CHUNK_MAX_SEGMENTS = 4096    # HS_CHUNK_MAX_SEGMENTS
CHUNK_MAX_TOKENS = 65536     # HS_CHUNK_MAX_TOKENS
COPY_MAX_PAGES = 4096        # HS_COPY_MAX_PAGES
PREFIX_MAX_GROUPS, PREFIX_MAX_TOKENS = 2048, 16384   # HS_PREFIX_MAX_*
ROTARY_MAX_DIMS, ROTARY_MAX_HEADS, ROTARY_MAX_PARTS = 256, 1024, 4   # HS_ROTARY_MAX_*
ROTARY_LAYOUTS = {"pairs": 0, "halves": 1}                        # HS_ROTARY_PAIRS, HS_ROTARY_HALVES
ROTARY_SCALINGS = {"none": 0, "linear": 1, "theta": 2, "ramp": 3}  # HS_ROTARY_NONE .. HS_ROTARY_RAMP


class RotaryConfig(ctypes.Structure):
    _fields_ = [("dims", ctypes.c_int32), ("scaling", ctypes.c_int32)] + \
               [(n, ctypes.c_double) for n in ("theta", "factor", "original_ctx", "beta_fast", "beta_slow", "magnitude")]


class RotaryPart(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_void_p), ("d_out", ctypes.c_void_p)] + \
               [(n, ctypes.c_int64) for n in ("in_stride_token", "in_stride_head", "out_stride_token", "out_stride_head")] + \
               [("heads", ctypes.c_int32), ("layout", ctypes.c_int32)]


_ROTARY_PART = struct.Struct("=QQqqqqii")   # RotaryPart in one call: each field set by itself takes longer than the kernel
assert _ROTARY_PART.size == ctypes.sizeof(RotaryPart)


_P = ctypes.c_void_p
_I = ctypes.c_int32
_L = ctypes.c_int64
_SIGS = {
    "hs_pool_config_check": [ctypes.POINTER(PoolConfig)],
    "hs_pool_init": [ctypes.POINTER(PoolConfig), ctypes.POINTER(_P), ctypes.POINTER(_P), _P, ctypes.POINTER(_P)],
    "hs_pool_destroy": [_P],
    "hs_request_set_pages": [_P, _I, _I, _I, _P, _P, _P, _P],
    "hs_hot_lease": [_P, _I, _I, _I, _P, _P],
    "hs_hot_release": [_P, _I, _P],
    "hs_append_rows": [_P, _I, _P, _P, _P, _P, _P],
    "hs_indexer_topk": [_P, _I, _I, _P, _P, _P, _P, _P, _P, _P],
    "hs_indexer_topk_noalloc": [_P, _I, _I, _P, _P, _P, _P, _P, _P],
    "hs_indexer_topk_fp8": [_P, _I, _I, _P, _P, _P, _P, _P, _P, _P],
    "hs_resolve_topk": [_P, _I, _I, _I, _P, _P, _P, _P, _P],
    "hs_replay_topk": [_P, _I, _I, _P, _P, _P, _P],
    "hs_sparse_mla_decode": [_P, _I, _I, _P, _P, ctypes.c_float, _P, _P, _P],
    "hs_offload_pages": [_P, _I, _P, _P, _P],
    "hs_append_quantized": [_P, _I, _I, _P, _P, _I, _P, _L, _P, _L, _P, _L, ctypes.c_float, _P],
    "hs_read_rows": [_P, _I, _I, _P, _P, _I, _P, _L, _P, _L, _P, _L, ctypes.c_float, _P],
    "hs_chunk_workspace": [_P, ctypes.POINTER(_L)],
    "hs_chunk_attention": [_P, _I, _I, _P, _P, _I, _P, _I, _P, _L, _L, ctypes.c_float, _P, _L, _L, _P, _P, _L, _P],
    "hs_rotary_steps": [ctypes.POINTER(RotaryConfig), _P, ctypes.POINTER(ctypes.c_float)],
    "hs_rotary_steps_of": [_I, _P, _P],
    "hs_rotary": [_P, _I, _P, _I, _P, ctypes.c_float, _I, _I, _I, _P, _P],
    "hs_fork_requests": [_P, _I, _P, _P, _P, _P, _P, _P],
    "hs_copy_pages": [_P, _I, _P, _P, _I, _P, _P, _I, _P],
    "hs_get_pages": [_P, _I, _P, _I, _I, _P, _P, _P, _P],
    "hs_prefix_workspace": [_P, _I, _I, _I, ctypes.POINTER(_L)],
    "hs_prefix_attention": [_P, _I, _I, _P, _P, _I, _P, _P, _I, _P, _I, _P, _L, _L, ctypes.c_float, _P, _L, _L, _P, _P, _L, _P],
    "hs_get_error": [_P, ctypes.POINTER(ctypes.c_int), _P],
    "hs_set_select_mode": [_P, _I],
    "hs_select_selftest": [_P, _I, _P, _P, _P],
    "hs_get_counters": [_P, ctypes.POINTER(Counters), _I, _P],
    "hs_link_probe": [_P, ctypes.c_int64, _I, _P, ctypes.c_int64, _P, _P],
    "hs_wait_selftest": [_P, _P],
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, args in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.hs_status_string.argtypes = [ctypes.c_int]
    lib.hs_status_string.restype = ctypes.c_char_p
    return lib


lib = _load()


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _current_device() -> int:
    import torch
    return torch.cuda.current_device() if torch.cuda.is_available() else -1


def _check(name: str, st: int) -> None:
    if st != 0:
        raise HisparseError(name, st)


_ARRAY_CODES = {ctypes.c_int32: "i", ctypes.c_int64: "q"}
assert all(array(code).itemsize == ctypes.sizeof(t) for t, code in _ARRAY_CODES.items())


def _host_array(values, ctype):
    """The address of values as an array of ctype, and what keeps it. A list of whole numbers is converted without a
    Python call for each (a context of 131,000 positions 26 us instead of 260); anything else as int() takes it."""
    if values is None:
        return None
    if not isinstance(values, (bytes, bytearray)):   # whose bytes array() would take for the elements'
        try:
            arr = array(_ARRAY_CODES[ctype], values)
            return arr.buffer_info()[0], arr
        except (TypeError, OverflowError):
            pass
    arr = (ctype * len(values))(*[int(v) for v in values])
    return ctypes.cast(arr, _P), arr


class _Torch:
    """What the prefill calls take from torch, looked up once: at a few microseconds of GPU
    time for a small call, the host's share of each call counts."""
    codes: dict = {}
    int32 = None
    int64 = None
    steps: tuple = ()
    raw_stream = None

    @classmethod
    def load(cls) -> None:
        import torch
        cls.int32, cls.int64 = torch.int32, torch.int64
        cls.steps = (torch.int64, torch.uint64)
        cls.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        cls.codes = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}

    @classmethod
    def load_once(cls) -> None:
        if not cls.codes:
            cls.load()


def _dtype(t) -> int:
    _Torch.load_once()
    code = _Torch.codes.get(t.dtype)
    if code is None:
        raise ValueError(f"element type {t.dtype}: bfloat16, float16 or float32 is wanted")
    return code


def _stream_of(stream, device: int) -> Optional[int]:
    """_stream() for a pool's device, without building a stream object."""
    if stream is None and _Torch.raw_stream is not None and device >= 0:
        return _Torch.raw_stream(device)
    return _stream(stream)


def _on(name: str, t, device: int) -> None:
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, the pool is on cuda:{device}")


def _ids(name: str, t, n: int, device: int) -> int:
    """The address of an int32 array of n elements."""
    if t.shape != (n,) or t.dtype is not _Torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 tensor of {n} elements is wanted")
    if t.get_device() != device:
        _on(name, t, device)
    return t.data_ptr()


def _values(name: str, t, n: int, width: int, dtype, device: int):
    """Address and row stride of [n, width] values whose last dimension is contiguous."""
    if t is None:
        return None, 0
    if t.shape != (n, width) or t.dtype is not dtype or t.stride(1) != 1:
        raise ValueError(f"{name}: a [{n}, {width}] tensor of the call's element type is wanted, last stride 1")
    if t.get_device() != device:
        _on(name, t, device)
    return t.data_ptr(), t.stride(0) if n > 1 else width


def rotary_steps(dims: int, theta: float, scaling: str = "none", factor: float = 1.0, original_ctx: float = 0.0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, magnitude: float = 0.0):
    """hs_rotary_steps: the steps [dims / 2] of Pool.rotary (an int64 tensor on the host, to be moved to the
    device once) for a scaling of ROTARY_SCALINGS, and the magnitude to give with them."""
    import torch
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling {scaling!r}: one of {', '.join(ROTARY_SCALINGS)} is wanted")
    cfg = RotaryConfig(dims, ROTARY_SCALINGS[scaling], theta, factor, original_ctx, beta_fast, beta_slow, magnitude)
    steps, m = torch.empty(max(dims, 0) // 2, dtype=torch.int64), ctypes.c_float(0.0)
    _check("hs_rotary_steps", lib.hs_rotary_steps(ctypes.byref(cfg), steps.data_ptr(), ctypes.byref(m)))
    return steps, m.value


def rotary_steps_of(frequencies):
    """hs_rotary_steps_of: the steps of frequencies of one's own, in radians per position."""
    import torch
    f = torch.as_tensor(frequencies, dtype=torch.float64, device="cpu").contiguous()
    if f.dim() != 1:
        raise ValueError("frequencies: one dimension is wanted")
    steps = torch.empty(f.numel(), dtype=torch.int64)
    _check("hs_rotary_steps_of", lib.hs_rotary_steps_of(f.numel(), f.data_ptr(), steps.data_ptr()))
    return steps


def config_ok(cfg: PoolConfig) -> bool:
    """hs_pool_config_check: whether hs_pool_init would accept this geometry (no GPU needed)."""
    return lib.hs_pool_config_check(ctypes.byref(cfg)) == 0


def link_probe(host_rows, row_bytes: int, src_rows, dst, stream=None) -> None:
    """hs_link_probe: copy dst[i] = host row src_rows[i] (single-row reads from a
    pinned, mapped host tensor), the access pattern of the resolver's miss copies."""
    _check("hs_link_probe", lib.hs_link_probe(_ptr(host_rows), host_rows.numel() * host_rows.element_size() // row_bytes,
                                              row_bytes, _ptr(src_rows), src_rows.numel(), _ptr(dst), _stream(stream)))


class Pool:
    """A HiSparse pool over caller-owned KV tensors, index caches and a pinned host pool."""

    def __init__(self, cfg: PoolConfig, kv_layers: Sequence, idx_layers: Sequence, host_kv):
        self.cfg = cfg
        self._keep = (list(kv_layers), list(idx_layers), host_kv)
        # the current device; without torch it is looked up by the first call that takes tensors
        self.device = _current_device() if sys.modules.get("torch") is not None else None
        kv = (_P * len(kv_layers))(*[_ptr(t) for t in kv_layers])
        ix = (_P * len(idx_layers))(*[_ptr(t) for t in idx_layers])
        handle = _P()
        _check("hs_pool_init", lib.hs_pool_init(ctypes.byref(cfg), kv, ix, _ptr(host_kv), ctypes.byref(handle)))
        self.handle = handle

    def close(self) -> None:
        if self.handle:
            _check("hs_pool_destroy", lib.hs_pool_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- host-side residency updates ------------------------------------------------
    def set_pages(self, req: int, first_page: int, block_table=None, idx_pages=None, host_pages=None,
                  stream=None) -> None:
        n = len(next(x for x in (block_table, idx_pages, host_pages) if x is not None))
        bt = _host_array(block_table, ctypes.c_int32)
        ip = _host_array(idx_pages, ctypes.c_int32)
        hp = _host_array(host_pages, ctypes.c_int64)
        _check("hs_request_set_pages", lib.hs_request_set_pages(
            self.handle, req, first_page, n, bt and bt[0], ip and ip[0], hp and hp[0], _stream(stream)))

    def hot_lease(self, req: int, group: int, pages, stream=None) -> None:
        arr = _host_array(pages, ctypes.c_int32)
        _check("hs_hot_lease", lib.hs_hot_lease(self.handle, req, group, len(pages), arr[0], _stream(stream)))

    def hot_release(self, req: int, stream=None) -> None:
        _check("hs_hot_release", lib.hs_hot_release(self.handle, req, _stream(stream)))

    # -- device hot path -------------------------------------------------------------
    def append_rows(self, req, pos, kv_rows, idx_keys, stream=None) -> None:
        _check("hs_append_rows", lib.hs_append_rows(self.handle, req.numel(), _ptr(req), _ptr(pos), _ptr(kv_rows),
                                                    _ptr(idx_keys), _stream(stream)))

    def indexer_topk(self, index_layer: int, req, limit, q, w, topk, scores=None, stream=None) -> None:
        _check("hs_indexer_topk", lib.hs_indexer_topk(self.handle, index_layer, req.numel(), _ptr(req), _ptr(limit),
                                                      _ptr(q), _ptr(w), _ptr(topk), _ptr(scores), _stream(stream)))

    def indexer_topk_fp8(self, index_layer: int, req, limit, q, w, topk, scores=None, stream=None) -> None:
        """FP8 keys (pool idx_format IDX_FP8): q e4m3 bytes, w fp32, scores nullable fp32."""
        _check("hs_indexer_topk_fp8", lib.hs_indexer_topk_fp8(self.handle, index_layer, req.numel(), _ptr(req),
                                                              _ptr(limit), _ptr(q), _ptr(w), _ptr(topk), _ptr(scores),
                                                              _stream(stream)))

    def indexer_topk_noalloc(self, index_layer: int, req, limit, q, w, topk, stream=None) -> None:
        """hs_indexer_topk with its score scratch in the library's fixed array, for
        callers that cannot allocate device memory (see include/hisparse.h)."""
        _check("hs_indexer_topk_noalloc", lib.hs_indexer_topk_noalloc(
            self.handle, index_layer, req.numel(), _ptr(req), _ptr(limit), _ptr(q), _ptr(w), _ptr(topk),
            _stream(stream)))

    def resolve_topk(self, group: int, step: int, req, topk, row_ids, plan=None, stream=None) -> None:
        _check("hs_resolve_topk", lib.hs_resolve_topk(self.handle, group, step, req.numel(), _ptr(req), _ptr(topk),
                                                      _ptr(row_ids), _ptr(plan), _stream(stream)))

    def replay_topk(self, group: int, req, topk, row_ids, stream=None) -> None:
        """Row ids of an already resolved selection, without touching the LRU state."""
        _check("hs_replay_topk", lib.hs_replay_topk(self.handle, group, req.numel(), _ptr(req), _ptr(topk),
                                                    _ptr(row_ids), _stream(stream)))

    def sparse_mla_decode(self, layer: int, q, row_ids, sm_scale: float, out, lse=None, stream=None) -> None:
        _check("hs_sparse_mla_decode", lib.hs_sparse_mla_decode(self.handle, layer, q.shape[0], _ptr(q),
                                                                _ptr(row_ids), float(sm_scale), _ptr(out),
                                                                _ptr(lse), _stream(stream)))

    def offload_pages(self, pool_pages, host_pages, stream=None) -> None:
        _check("hs_offload_pages", lib.hs_offload_pages(self.handle, pool_pages.numel(), _ptr(pool_pages),
                                                        _ptr(host_pages), _stream(stream)))

    # -- prefill and dense decode, one layer at a time ---------------------------------
    def _device(self) -> int:
        if self.device is None:
            self.chunk_workspace_bytes()     # refused unless the pool's device is the current one
            self.device = _current_device()
        return self.device

    def _cache_args(self, req, pos, latent, rope, keys):
        first = latent if latent is not None else rope if rope is not None else keys
        if first is None:
            raise ValueError("none of latent, rope and keys is given")
        code, dtype, n, dev = _dtype(first), first.dtype, req.shape[0], self._device()
        return (n, _ids("req", req, n, dev), _ids("pos", pos, n, dev), code,
                *_values("latent", latent, n, 512, dtype, dev), *_values("rope", rope, n, 64, dtype, dev),
                *_values("keys", keys, n, 128, dtype, dev))

    def append_quantized(self, layer: int, req, pos, latent=None, rope=None, keys=None, key_scale: float = 1.0,
                         stream=None) -> None:
        """Quantise new rows of one layer into the cache: latent [n, 512] and rope [n, 64]
        (both or neither), index keys [n, 128]; bf16, fp16 or fp32, rows may be strided.
        key_scale: the step of int8 index keys."""
        _check("hs_append_quantized", lib.hs_append_quantized(
            self.handle, layer, *self._cache_args(req, pos, latent, rope, keys), key_scale,
            _stream_of(stream, self.device)))

    def read_rows(self, layer: int, req, pos, latent=None, rope=None, keys=None, key_scale: float = 1.0,
                  stream=None) -> None:
        """Read cached positions of one layer back into latent [n, 512], rope [n, 64] and
        keys [n, 128] (any of them), in their element type."""
        _check("hs_read_rows", lib.hs_read_rows(
            self.handle, layer, *self._cache_args(req, pos, latent, rope, keys), key_scale,
            _stream_of(stream, self.device)))

    def chunk_workspace_bytes(self) -> int:
        """Bytes of device workspace that chunk_attention needs, whatever the call's sizes."""
        n = _L(0)
        _check("hs_chunk_workspace", lib.hs_chunk_workspace(self.handle, ctypes.byref(n)))
        return n.value

    def chunk_attention(self, layer: int, seg_req, seg_start, limit, q, sm_scale: float, out, work, lse=None,
                        stream=None) -> None:
        """Attention of new tokens over every cached row below their limits. Segment i is the
        tokens [seg_start[i], seg_start[i + 1]) of request seg_req[i]; limit [n]; q [n, H, 576]
        and out [n, H, 512] bf16 or fp16, the last dimension contiguous; lse [n, H] fp32;
        work: chunk_workspace_bytes() bytes that no overlapping call uses."""
        _check("hs_chunk_attention", lib.hs_chunk_attention(
            self.handle, layer, *self._attention_args(seg_req, seg_start, limit, q, sm_scale, out, work, lse, stream)))

    def _attention_args(self, seg_req, seg_start, limit, q, sm_scale, out, work, lse, stream):
        code, n, segs, heads, dev = _dtype(q), limit.shape[0], seg_req.shape[0], self.cfg.n_heads, self._device()
        if q.shape != (n, heads, 576) or out.shape != (n, heads, 512) or out.dtype is not q.dtype:
            raise ValueError(f"q [{n}, {heads}, 576] and out [{n}, {heads}, 512] of one type are wanted")
        qs, os = q.stride(), out.stride()
        if qs[2] != 1 or os[2] != 1:
            raise ValueError("q and out: a contiguous last dimension is wanted")
        if lse is not None and (lse.shape != (n, heads) or _dtype(lse) != FP32 or not lse.is_contiguous()):
            raise ValueError(f"lse: a contiguous fp32 [{n}, {heads}] tensor is wanted")
        if not work.is_contiguous():
            raise ValueError("work: a contiguous tensor is wanted")
        if q.get_device() != dev or out.get_device() != dev or work.get_device() != dev or \
                (lse is not None and lse.get_device() != dev):
            raise ValueError(f"q, out, lse or work is not on the pool's device, cuda:{dev}")
        return (segs, _ids("seg_req", seg_req, segs, dev), _ids("seg_start", seg_start, segs + 1, dev),
                n, _ids("limit", limit, n, dev), code, q.data_ptr(), qs[0] if n > 1 else heads * 576, qs[1], sm_scale,
                out.data_ptr(), os[0] if n > 1 else heads * 512, os[1], None if lse is None else lse.data_ptr(),
                work.data_ptr(), work.numel() * work.element_size(), _stream_of(stream, dev))

    # -- requests that share a prompt ---------------------------------------------------
    def rotary(self, pos, steps, parts, magnitude: float = 1.0, inverse: bool = False, stream=None) -> None:
        """Rotary positions of up to four tensors of the same tokens in one launch. pos [n] int32; steps
        [dims / 2] from rotary_steps, on the device; parts: (x, out, layout) with x and out [n, heads, dims]
        or [n, dims] of one type, views of the rotated dims with a contiguous last one, out x itself for
        in place; layout "pairs" or "halves". inverse turns backwards (the transpose)."""
        k = len(parts)
        if not 0 < k <= ROTARY_MAX_PARTS:
            raise ValueError(f"1 to {ROTARY_MAX_PARTS} parts are wanted")
        first = parts[0][0]
        code, dtype, n, dev = _dtype(first), first.dtype, pos.shape[0], self._device()
        dims = first.shape[-1]
        packed = bytearray(_ROTARY_PART.size * k)
        at = 0
        for x, out, layout in parts:
            shape, xs, os = x.shape, x.stride(), out.stride()
            if out.shape != shape or shape[0] != n or shape[-1] != dims:
                raise ValueError(f"x and out [{n}, heads, {dims}] or [{n}, {dims}] of one shape are wanted")
            if x.dtype is not dtype or out.dtype is not dtype:
                raise ValueError("all parts of one element type are wanted")
            if xs[-1] != 1 or os[-1] != 1:
                raise ValueError("x and out: a contiguous last dimension is wanted")
            if x.get_device() != dev or out.get_device() != dev:
                raise ValueError(f"x or out is not on the pool's device, cuda:{dev}")
            if layout not in ROTARY_LAYOUTS:
                raise ValueError(f"layout {layout!r}: pairs or halves is wanted")
            if len(xs) == 3:
                heads, xh, oh = shape[1], xs[1], os[1]
                if heads == 1:
                    xh = oh = dims
            elif len(xs) == 2:
                heads, xh, oh = 1, dims, dims
            else:
                raise ValueError(f"x and out [{n}, heads, {dims}] or [{n}, {dims}] are wanted")
            xt, ot = (xs[0], os[0]) if n > 1 else (dims, dims)
            _ROTARY_PART.pack_into(packed, at, x.data_ptr(), out.data_ptr(), xt, xh, ot, oh, heads, ROTARY_LAYOUTS[layout])
            at += _ROTARY_PART.size
        if steps.shape != (dims // 2,) or steps.dtype not in _Torch.steps or not steps.is_contiguous():
            raise ValueError(f"steps: a contiguous int64 tensor of {dims // 2} elements is wanted")
        if steps.get_device() != dev:
            _on("steps", steps, dev)
        _check("hs_rotary", lib.hs_rotary(self.handle, n, _ids("pos", pos, n, dev), dims, steps.data_ptr(), magnitude,
                                          1 if inverse else 0, code, k, bytes(packed), _stream_of(stream, dev)))

    def fork_requests(self, src, dst, length, tail_pages, tail_idx_pages=None, stream=None) -> None:
        """Begin requests dst[i] with the first length[i] positions of src[i]: whole pages shared, the rows of
        a last, partly filled page copied into tail_pages[i] and tail_idx_pages[i]. All [n] int32 on the device."""
        _Torch.load_once()
        n, dev = src.shape[0], self._device()
        _check("hs_fork_requests", lib.hs_fork_requests(
            self.handle, n, _ids("src", src, n, dev), _ids("dst", dst, n, dev), _ids("length", length, n, dev),
            _ids("tail_pages", tail_pages, n, dev),
            None if tail_idx_pages is None else _ids("tail_idx_pages", tail_idx_pages, n, dev), _stream_of(stream, dev)))

    def copy_pages(self, src=None, dst=None, idx_src=None, idx_dst=None, remap: bool = False, stream=None) -> None:
        """Copy pool pages src[i] -> dst[i] in every layer and index pages idx_src[i] -> idx_dst[i] in every
        indexer layer (int32 on the device, either kind may be left out); remap: move them, every table entry
        that names src[i] naming dst[i] afterwards."""
        if (src is None) != (dst is None) or (idx_src is None) != (idx_dst is None):
            raise ValueError("sources and destinations: both or neither are wanted")
        dev = self._device()
        _Torch.load_once()
        n = m = 0
        at = to = idx_at = idx_to = None
        if src is not None:
            n = src.shape[0]
            at, to = _ids("src", src, n, dev), _ids("dst", dst, n, dev)
        if idx_src is not None:
            m = idx_src.shape[0]
            idx_at, idx_to = _ids("idx_src", idx_src, m, dev), _ids("idx_dst", idx_dst, m, dev)
        _check("hs_copy_pages", lib.hs_copy_pages(self.handle, n, at, to, m, idx_at, idx_to, 1 if remap else 0,
                                                  _stream_of(stream, dev)))

    def prefix_workspace_bytes(self, n_tokens: int, n_segments: int, n_groups: int) -> int:
        """Bytes of device workspace that prefix_attention needs for a call of at most these sizes."""
        n = _L(0)
        _check("hs_prefix_workspace", lib.hs_prefix_workspace(self.handle, n_tokens, n_segments, n_groups, ctypes.byref(n)))
        return n.value

    def prefix_attention(self, layer: int, group_start, group_len, seg_req, seg_start, limit, q, sm_scale: float, out, work,
                         lse=None, stream=None) -> None:
        """chunk_attention for requests that share their first positions: group i is the segments
        [group_start[i], group_start[i + 1]), whose requests hold the same rows at positions [0, group_len[i]);
        these are read and multiplied once for the tokens of all of them. work: prefix_workspace_bytes() bytes."""
        args = self._attention_args(seg_req, seg_start, limit, q, sm_scale, out, work, lse, stream)
        groups, dev = group_len.shape[0], self._device()
        _check("hs_prefix_attention", lib.hs_prefix_attention(
            self.handle, layer, groups, _ids("group_start", group_start, groups + 1, dev),
            _ids("group_len", group_len, groups, dev), *args))

    def get_pages(self, req, first_page: int, block_table=None, idx_pages=None, host_pages=None, stream=None) -> None:
        """Read table entries [first_page, first_page + n_pages) of requests req [n] into block_table and
        idx_pages (int32) and host_pages (int64), each [n, n_pages] on the device, any of them left out."""
        first = block_table if block_table is not None else idx_pages if idx_pages is not None else host_pages
        if first is None:
            raise ValueError("none of block_table, idx_pages and host_pages is given")
        _Torch.load_once()
        n, dev, shape = req.shape[0], self._device(), first.shape
        if len(shape) != 2 or shape[0] != n:
            raise ValueError(f"outputs [{n}, pages] are wanted")

        def table(name, t, dtype):
            if t is None:
                return None
            if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
                raise ValueError(f"{name}: a contiguous {dtype} tensor [{n}, pages] is wanted, of one shape with the others")
            if t.get_device() != dev:
                _on(name, t, dev)
            return t.data_ptr()
        _check("hs_get_pages", lib.hs_get_pages(
            self.handle, n, _ids("req", req, n, dev), first_page, shape[1], table("block_table", block_table, _Torch.int32),
            table("idx_pages", idx_pages, _Torch.int32), table("host_pages", host_pages, _Torch.int64), _stream_of(stream, dev)))

    # -- status --------------------------------------------------------------------
    def get_error(self, stream=None) -> int:
        v = ctypes.c_int(0)
        _check("hs_get_error", lib.hs_get_error(self.handle, ctypes.byref(v), _stream(stream)))
        return v.value

    def set_select_mode(self, mode: int) -> None:
        """hs_set_select_mode: SELECT_LOCAL keeps the top-K selection off grid-wide waits."""
        _check("hs_set_select_mode", lib.hs_set_select_mode(self.handle, mode))

    def select_selftest(self, limit, topk, stream=None) -> None:
        """hs_select_selftest: the grid-wide selection with one CTA per token withholding
        its arrivals, so the others time out (HS_ERR_TIMEOUT, half-used scratch)."""
        _check("hs_select_selftest", lib.hs_select_selftest(self.handle, limit.numel(), _ptr(limit), _ptr(topk),
                                                            _stream(stream)))

    def wait_selftest(self, stream=None) -> None:
        """hs_wait_selftest: a bounded device wait that runs out (HS_ERR_TIMEOUT)."""
        _check("hs_wait_selftest", lib.hs_wait_selftest(self.handle, _stream(stream)))

    def raise_on_device_error(self, stream=None) -> None:
        st = self.get_error(stream)
        if st:
            raise HisparseError("device", st)

    def counters(self, reset: bool = False, stream=None) -> Counters:
        c = Counters()
        _check("hs_get_counters", lib.hs_get_counters(self.handle, ctypes.byref(c), int(reset), _stream(stream)))
        return c
