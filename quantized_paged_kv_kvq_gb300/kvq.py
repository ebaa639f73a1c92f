"""Python binding of libkvq.so (argument marshalling only).

Every function here has the name of the C entry point it calls and does
nothing but turn torch tensors into pointers and sizes; all work runs in the
library's CUDA kernels on the current torch stream.  The library must have
been built (quantized_paged_kv_kvq_gb300.build); importing this module
without it raises, and there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

FMT = {"int8": 1, "fp8_e4m3": 2, "fp8_e5m2": 3, "int4_asym": 4, "uint8_asym": 5, "bf16": 6}
ASYM = ("int4_asym", "uint8_asym")
FLAG_VARNORM_ROTATE = 1
STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARGUMENT", 2: "KVQ_ERR_UNSUPPORTED",
          3: "KVQ_ERR_WORKSPACE", 4: "KVQ_ERR_CUDA"}
DEVERR_SLOT_RANGE = 1
DEVERR_BLOCK_RANGE = 2
DEVERR_CONTEXT_RANGE = 4
DEVERR_COMBINE = 8
DEVERR_TIMEOUT = 16
DEVERR_CLASS_RANGE = 32
DEVERR_QUERY_RANGE = 64
DEVERR_FREE_BLOCKS = 128
DEVERR_TOKENS = 256
DEVERR_POSITION = 512
ROPE_KIND = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class KvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class _CacheDesc(ctypes.Structure):
    _fields_ = [("k_fmt", ctypes.c_int32), ("v_fmt", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("k_meta", ctypes.c_void_p),
                ("v_meta", ctypes.c_void_p), ("signs", ctypes.c_void_p),
                ("k_head_scales", ctypes.c_void_p), ("v_head_scales", ctypes.c_void_p)]


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("amplitude", ctypes.c_double)]


class _RopeDesc(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("num_positions", ctypes.c_int64)]


_P = ctypes.c_void_p
_I32, _I64, _F32, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_F64 = ctypes.c_double
_DESC = ctypes.POINTER(_CacheDesc)
_ROPE = ctypes.POINTER(_RopeDesc)

# name -> (restype, argtypes)
SIGNATURES = {
    "kvq_write_cache": (_I32, [_DESC, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P]),
    "kvq_decode_workspace_size": (_I32, [_DESC, _I32, _I32, _I32, ctypes.POINTER(_SZ)]),
    "kvq_decode_workspace_size_ex": (_I32, [_DESC, _I32, _I32, _I32, _I32, ctypes.POINTER(_SZ)]),
    "kvq_paged_decode": (_I32, [_DESC, _P, _P, _P, _P, _I32, _I32, _P, _I32, _P, _I32, _F32, _P,
                                _SZ, _P]),
    "kvq_paged_decode_ex": (_I32, [_DESC, _P, _P, _P, _P, _I32, _I32, _P, _I32, _P, _I32, _F32,
                                   _I32, _P, _SZ, _P]),
    "kvq_decode_append": (_I32, [_DESC, _P, _P, _P, _P, _I64, _I64, _P, _P, _I32, _I32, _P, _I32,
                                 _P, _I32, _F32, _I32, _P, _SZ, _P]),
    "kvq_paged_decode_static": (_I32, [_DESC, _P, _P, _P, _P, _I32, _I32, _P, _I32, _P, _I32,
                                       _F32, _I32, _P]),
    "kvq_decode_mixed": (_I32, [_DESC, _I32, ctypes.POINTER(_P), ctypes.POINTER(_P), _P, _P, _P,
                                _I64, _I64, _P, _P, _I32, _I32, _P, _I32, _P, _I32, _F32, _I32,
                                _P, _SZ, _P]),
    "kvq_paged_decode_static_capacity": (_SZ, []),
    "kvq_plan_step": (_I32, [_P, _P, _I32, _P, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _I64, _P,
                             _P, _P, _P]),
    "kvq_rope_table": (_I32, [_P, _I64, _I32, _F64, ctypes.POINTER(_RopeScaling), _P]),
    "kvq_norm_rope": (_I32, [_ROPE, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I32, _I32,
                             _P]),
    "kvq_norm_rope_write": (_I32, [_ROPE, _DESC, _P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                                   _P, _P, _I64, _I32, _P]),
    "kvq_decode_window": (_I32, [_DESC, _P, _P, _P, _P, _I64, _I64, _P, _P, _I32, _I32, _P, _I32,
                                 _P, _I32, _F32, _I32, _I32, _I32, _P, _SZ, _P]),
    "kvq_prefill_workspace_size": (_I32, [_DESC, _I32, _I32, _I64, _I32, _I32,
                                          ctypes.POINTER(_SZ)]),
    "kvq_paged_prefill": (_I32, [_DESC, _P, _P, _P, _P, _P, _I32, _I64, _I32, _I32, _P, _I32, _P,
                                 _I32, _F32, _I32, _I32, _P, _SZ, _P]),
    "kvq_hadamard": (_I32, [_P, _I32, _I64, _I32, _P, _I32, _P]),
    "kvq_calibrate_scale": (_I32, [_P, _I64, _F32, _P, _P]),
    "kvq_calibrate_head_scales": (_I32, [_P, _I64, _I32, _I32, _I64, _F32, _P, _P]),
    "kvq_debug_arm_wait_timeout": (_I32, [_I32, _I32, _I32]),
    "kvq_get_device_error": (_I32, [_P, ctypes.POINTER(ctypes.c_uint32)]),
    "kvq_status_string": (ctypes.c_char_p, [_I32]),
    "kvq_version": (ctypes.c_char_p, []),
}

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libkvq.so (once) and declare its entry points; raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m quantized_paged_kv_kvq_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        raise KvqError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


@dataclass
class KVCache:
    """One layer's paged cache: caller-owned device tensors + description.

    k_cache / v_cache: uint8 [num_blocks, block_size, num_kv_heads, row_bytes]
    k_meta / v_meta:   fp16 [num_blocks, num_kv_heads, F, block_size] (asymmetric formats)
    signs:             int8 [head_dim] of +-1 (KVarN rotation) or None

    The tensors may hold more blocks than num_blocks.
    """
    k_fmt: str
    v_fmt: str
    num_kv_heads: int
    head_dim: int
    block_size: int
    num_blocks: int
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_meta: Optional[torch.Tensor] = None
    v_meta: Optional[torch.Tensor] = None
    k_scale: float = 1.0
    v_scale: float = 1.0
    varnorm_rotate: bool = False
    signs: Optional[torch.Tensor] = None
    k_head_scales: Optional[torch.Tensor] = None  # fp32 [num_kv_heads] (symmetric K)
    v_head_scales: Optional[torch.Tensor] = None  # fp32 [num_kv_heads] (symmetric V)

    def desc(self) -> _CacheDesc:
        ptr = lambda t: None if t is None else t.data_ptr()
        return _CacheDesc(FMT[self.k_fmt], FMT[self.v_fmt], self.num_kv_heads, self.head_dim,
                          self.block_size, self.num_blocks,
                          FLAG_VARNORM_ROTATE if self.varnorm_rotate else 0,
                          float(self.k_scale), float(self.v_scale), ptr(self.k_meta),
                          ptr(self.v_meta), ptr(self.signs), ptr(self.k_head_scales),
                          ptr(self.v_head_scales))


def row_bytes(fmt: str, head_dim: int) -> int:
    return head_dim // 2 if fmt == "int4_asym" else 2 * head_dim if fmt == "bf16" else head_dim


def meta_fields(fmt: str, varnorm_rotate: bool) -> int:
    if fmt in ASYM:
        return 3 if varnorm_rotate else 2
    return 0


def alloc_kv_cache(k_fmt, v_fmt, num_blocks, block_size, num_kv_heads, head_dim,
                   k_scale=1.0, v_scale=1.0, varnorm_rotate=False, signs=None,
                   device="cuda", fill: Optional[int] = None) -> KVCache:
    """Allocate (with torch) the device tensors of a cache; `fill` poisons them."""
    def codes(fmt):
        t = torch.empty((num_blocks, block_size, num_kv_heads, row_bytes(fmt, head_dim)),
                        dtype=torch.uint8, device=device)
        if fill is not None:
            t.fill_(fill)
        return t

    def meta(fmt):
        nf = meta_fields(fmt, varnorm_rotate)
        if not nf:
            return None
        t = torch.empty((num_blocks, num_kv_heads, nf, block_size), dtype=torch.float16,
                        device=device)
        if fill is not None:
            t.view(torch.int16).fill_(fill * 0x101 - (0x10000 if fill * 0x101 >= 0x8000 else 0))
        return t

    return KVCache(k_fmt, v_fmt, num_kv_heads, head_dim, block_size, num_blocks, codes(k_fmt),
                   codes(v_fmt), meta(k_fmt), meta(v_fmt), k_scale, v_scale, varnorm_rotate,
                   signs)


def kvq_write_cache(cache: KVCache, key: torch.Tensor, value: torch.Tensor,
                    slot_mapping: torch.Tensor, stream=None) -> None:
    """Quantize key/value (bf16 [T, Hkv, D], token stride free) into the cache."""
    lib = load_library()
    assert key.dtype == torch.bfloat16 and value.dtype == torch.bfloat16
    assert slot_mapping.dtype == torch.int64
    t = key.shape[0]
    d = cache.desc()
    st = lib.kvq_write_cache(ctypes.byref(d), _ptr(cache.k_cache), _ptr(cache.v_cache), _ptr(key),
                             _ptr(value), key.stride(0), value.stride(0), _ptr(slot_mapping), t,
                             _stream(stream))
    _check(st, "kvq_write_cache")


def kvq_decode_workspace_size(cache: KVCache, num_seqs: int, num_q_heads: int,
                              max_context_len: int, num_ctas: int = 0) -> int:
    lib = load_library()
    n = ctypes.c_size_t(0)
    d = cache.desc()
    st = lib.kvq_decode_workspace_size_ex(ctypes.byref(d), num_seqs, num_q_heads,
                                          max_context_len, num_ctas, ctypes.byref(n))
    _check(st, "kvq_decode_workspace_size")
    return int(n.value)


def _decode_call(fn_name, cache, query, out, block_table, context_lens, max_context_len,
                 sm_scale, workspace, num_ctas, stream):
    lib = load_library()
    assert query.dtype == torch.bfloat16 and out.dtype == torch.bfloat16
    assert query.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and context_lens.dtype == torch.int32
    assert block_table.is_contiguous()
    s, hq, _ = query.shape
    d = cache.desc()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = getattr(lib, fn_name)(ctypes.byref(d), _ptr(cache.k_cache), _ptr(cache.v_cache),
                               _ptr(out), _ptr(query), s, hq, _ptr(block_table),
                               block_table.shape[1], _ptr(context_lens), max_context_len,
                               float(sm_scale), num_ctas, _ptr(workspace), ws_bytes,
                               _stream(stream))
    _check(st, fn_name)
    return out


def kvq_paged_decode(cache: KVCache, query: torch.Tensor, out: torch.Tensor,
                     block_table: torch.Tensor, context_lens: torch.Tensor, max_context_len: int,
                     sm_scale: float, workspace: Optional[torch.Tensor] = None,
                     num_ctas: int = 0, stream=None) -> torch.Tensor:
    """out[s, h] = softmax(sm_scale q k^T) v over the paged cache (bf16 [S, Hq, D])."""
    return _decode_call("kvq_paged_decode_ex", cache, query, out, block_table, context_lens,
                        max_context_len, sm_scale, workspace, num_ctas, stream)


def kvq_decode_append(cache: KVCache, new_key: torch.Tensor, new_value: torch.Tensor,
                      query: torch.Tensor, out: torch.Tensor, block_table: torch.Tensor,
                      context_lens: torch.Tensor, max_context_len: int, sm_scale: float,
                      workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                      stream=None) -> torch.Tensor:
    """One decode step in one launch: row s of new_key / new_value (bf16 [S, Hkv, D],
    sequence stride free) is quantized into the cache at position context_lens[s] - 1,
    then out = the paged decode over the context including it."""
    lib = load_library()
    assert new_key.dtype == torch.bfloat16 and new_value.dtype == torch.bfloat16
    assert query.dtype == torch.bfloat16 and out.dtype == torch.bfloat16
    assert query.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and context_lens.dtype == torch.int32
    assert block_table.is_contiguous()
    s, hq, _ = query.shape
    d = cache.desc()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.kvq_decode_append(ctypes.byref(d), _ptr(cache.k_cache), _ptr(cache.v_cache),
                               _ptr(new_key), _ptr(new_value), new_key.stride(0),
                               new_value.stride(0), _ptr(out), _ptr(query), s, hq,
                               _ptr(block_table), block_table.shape[1], _ptr(context_lens),
                               max_context_len, float(sm_scale), num_ctas, _ptr(workspace),
                               ws_bytes, _stream(stream))
    _check(st, "kvq_decode_append")
    return out


def kvq_decode_mixed(classes, seq_class: torch.Tensor, query: torch.Tensor, out: torch.Tensor,
                     block_table: torch.Tensor, context_lens: torch.Tensor, max_context_len: int,
                     sm_scale: float, workspace: Optional[torch.Tensor] = None,
                     num_ctas: int = 0, new_key: Optional[torch.Tensor] = None,
                     new_value: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode (or, with new_key / new_value, the fused append step) over a cache
    of several page classes: `classes` is a list of KVCache, one pool per page
    size; seq_class (uint8 [S]) names each sequence's class, and block_table
    row s holds block ids of that class's pool."""
    lib = load_library()
    assert seq_class.dtype == torch.uint8 and seq_class.is_contiguous()
    assert query.dtype == torch.bfloat16 and out.dtype == torch.bfloat16
    assert query.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and context_lens.dtype == torch.int32
    assert block_table.is_contiguous()
    n = len(classes)
    descs = (_CacheDesc * n)(*[c.desc() for c in classes])
    kcs = (ctypes.c_void_p * n)(*[c.k_cache.data_ptr() for c in classes])
    vcs = (ctypes.c_void_p * n)(*[c.v_cache.data_ptr() for c in classes])
    s, hq, _ = query.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ks = 0 if new_key is None else new_key.stride(0)
    vs = 0 if new_value is None else new_value.stride(0)
    st = lib.kvq_decode_mixed(descs, n, kcs, vcs, _ptr(seq_class), _ptr(new_key),
                              _ptr(new_value), ks, vs, _ptr(out), _ptr(query), s, hq,
                              _ptr(block_table), block_table.shape[1], _ptr(context_lens),
                              max_context_len, float(sm_scale), num_ctas, _ptr(workspace),
                              ws_bytes, _stream(stream))
    _check(st, "kvq_decode_mixed")
    return out


def kvq_paged_decode_static(cache: KVCache, query: torch.Tensor, out: torch.Tensor,
                            block_table: torch.Tensor, context_lens: torch.Tensor,
                            max_context_len: int, sm_scale: float, num_ctas: int = 0,
                            stream=None) -> torch.Tensor:
    """kvq_paged_decode for callers that cannot allocate: the split-K scratch is
    the library's own fixed array (kvq_paged_decode_static_capacity() bytes)
    instead of a workspace tensor.  Calls that overlap on the GPU race on it."""
    lib = load_library()
    assert query.dtype == torch.bfloat16 and out.dtype == torch.bfloat16
    assert query.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and context_lens.dtype == torch.int32
    assert block_table.is_contiguous()
    s, hq, _ = query.shape
    d = cache.desc()
    st = lib.kvq_paged_decode_static(ctypes.byref(d), _ptr(cache.k_cache), _ptr(cache.v_cache),
                                     _ptr(out), _ptr(query), s, hq, _ptr(block_table),
                                     block_table.shape[1], _ptr(context_lens), max_context_len,
                                     float(sm_scale), num_ctas, _stream(stream))
    _check(st, "kvq_paged_decode_static")
    return out


def kvq_paged_decode_static_capacity() -> int:
    return int(load_library().kvq_paged_decode_static_capacity())


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


# The calls below take a few microseconds on the GPU, and these checks run before each
# of them: one device query per call, then plain comparisons.  torch's own shortcuts to
# the current device and its stream's handle serve where this torch has them (2.9 and
# 2.11 do: 0.1 us each, where the public calls take 0.2 and 1.1), else the public calls.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                       or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))


def _device_of(name: str, t: torch.Tensor) -> int:
    """The current CUDA device, which t must be on."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")
    return dev


def _int32(**values) -> None:
    """Refuses numbers that the C call's 32-bit arguments do not hold (ctypes would cut them)."""
    for name, v in values.items():
        if not -0x80000000 <= v <= 0x7fffffff:
            raise ValueError(f"{name} must fit 32 bits, got {v}")


def _tensors(dev: int, *specs) -> None:
    """Each (name, tensor, dtype, shape): a contiguous tensor of CUDA device dev."""
    for name, t, dtype, shape in specs:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on CUDA "
                             f"device {dev}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _rows(dev: int, name: str, t: torch.Tensor, shape) -> int:
    """Checks bf16 [T, heads, D] rows with a free token stride; returns that stride."""
    if t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a bf16 tensor of shape {tuple(shape)} on CUDA device {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    n, heads, d = shape
    s0, s1, s2 = t.stride()
    if ((s2 != 1 and d > 1) or (s1 != d and heads > 1)) and t.numel():
        raise ValueError(f"{name}: heads and elements must be contiguous, got strides {t.stride()}")
    # one token: any stride serves, and torch may report one that is too small
    return s0 if n > 1 else (heads * d + 7) // 8 * 8


def _pool(dev: int, name: str, t: torch.Tensor, dtype, blocks: int, a: int, b: int, c: int) -> None:
    """Checks a cache's contiguous tensor [blocks or more, a, b, c] of CUDA device dev."""
    shape = t.shape
    if (t.dtype is not dtype or len(shape) != 4 or shape[0] < blocks or shape != (shape[0], a, b, c)
            or t.get_device() != dev or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {(blocks, a, b, c)} on CUDA device {dev}, "
                         f"got {t.dtype} {tuple(shape)} with strides {t.stride()} on {t.device}")


def _cache_desc(dev: int, cache: KVCache) -> _CacheDesc:
    """The cache's description, once its tensors are what it says: the kernels write and
    read through them, and see nothing but addresses."""
    c, rot = cache, cache.varnorm_rotate
    blocks, bs, hkv, d = c.num_blocks, c.block_size, c.num_kv_heads, c.head_dim
    _pool(dev, "k_cache", c.k_cache, torch.uint8, blocks, bs, hkv, row_bytes(c.k_fmt, d))
    _pool(dev, "v_cache", c.v_cache, torch.uint8, blocks, bs, hkv, row_bytes(c.v_fmt, d))
    if c.k_fmt in ASYM:
        _need(c.k_meta is not None, "k_meta is missing: rows of this format have fields")
        _pool(dev, "k_meta", c.k_meta, torch.float16, blocks, hkv, 3 if rot else 2, bs)
    if c.v_fmt in ASYM:
        _need(c.v_meta is not None, "v_meta is missing: rows of this format have fields")
        _pool(dev, "v_meta", c.v_meta, torch.float16, blocks, hkv, 3 if rot else 2, bs)
    if rot and c.signs is not None:
        _tensors(dev, ("signs", c.signs, torch.int8, (d,)))
    if c.k_head_scales is not None:
        _tensors(dev, ("k_head_scales", c.k_head_scales, torch.float32, (hkv,)))
    if c.v_head_scales is not None:
        _tensors(dev, ("v_head_scales", c.v_head_scales, torch.float32, (hkv,)))
    return c.desc()


def _workspace(dev: int, workspace: Optional[torch.Tensor]) -> int:
    if workspace is None:
        return 0
    _need(workspace.get_device() == dev and workspace.is_contiguous(),
          "workspace must be contiguous, on the current CUDA device")
    return workspace.numel() * workspace.element_size()


def _raw_stream(dev: int, stream) -> int:
    """A stream's handle (the current one's if None)."""
    return _current_raw_stream(dev) if stream is None else stream.cuda_stream


def _address(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def kvq_plan_step(context_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
                  free_blocks: torch.Tensor, free_range: torch.Tensor, block_size: int,
                  num_blocks: int, slot_mapping: torch.Tensor, positions: torch.Tensor,
                  context_lens_out: torch.Tensor, cu_new: torch.Tensor,
                  free_range_out: torch.Tensor, stream=None) -> None:
    """Plan one serving step on the GPU: context_lens and new_lens (int32 [S]) give the
    tokens cached and added; block_table (int32 [S, W]) gets the free blocks its new pages
    need (free_blocks int32 [F], entries free_range[0]..free_range[1]-1), slot_mapping
    (int64 [T]) and positions (int32 [T]) describe the packed new tokens (slot -1 behind
    the last), context_lens_out (int32 [S]), cu_new (int32 [S+1]) and free_range_out
    (int32 [2]) the state after the step."""
    s, t, i32 = context_lens.numel(), slot_mapping.numel(), torch.int32
    width, free = block_table.shape[-1], free_blocks.numel()
    _int32(block_size=block_size, num_blocks=num_blocks, free_blocks=free)
    dev = _device_of("slot_mapping", slot_mapping)
    _tensors(dev, ("context_lens", context_lens, i32, (s,)), ("new_lens", new_lens, i32, (s,)),
             ("block_table", block_table, i32, (s, width)), ("free_blocks", free_blocks, i32, (free,)),
             ("free_range", free_range, i32, (2,)), ("slot_mapping", slot_mapping, torch.int64, (t,)),
             ("positions", positions, i32, (t,)), ("context_lens_out", context_lens_out, i32, (s,)),
             ("cu_new", cu_new, i32, (s + 1,)), ("free_range_out", free_range_out, i32, (2,)))
    st = load_library().kvq_plan_step(
        context_lens.data_ptr(), new_lens.data_ptr(), s, block_table.data_ptr(), width, block_size,
        num_blocks, free_blocks.data_ptr(), free, free_range.data_ptr(), slot_mapping.data_ptr(),
        positions.data_ptr(), t, context_lens_out.data_ptr(), cu_new.data_ptr(),
        free_range_out.data_ptr(), _raw_stream(dev, stream))
    _check(st, "kvq_plan_step")


@dataclass
class RopeScaling:
    """How a rotation table is stretched (kvq_rope_kind in include/kvq.h): kind "linear",
    "ntk", "yarn" or "bands" by `factor`; original_len, low and high for the last two."""
    kind: str
    factor: float = 1.0
    original_len: float = 1.0
    low: float = 1.0
    high: float = 2.0
    amplitude: float = 1.0


def kvq_rope_table(table: torch.Tensor, base: float, scaling: Optional[RopeScaling] = None,
                   stream=None) -> torch.Tensor:
    """table (fp32 [positions, rot_dim / 2, 2]) <- cos and sin of every position and pair."""
    _need(table.dim() == 3, "table must have shape (positions, rot_dim / 2, 2)")
    n, pairs = table.shape[:2]
    dev = _device_of("table", table)
    _tensors(dev, ("table", table, torch.float32, (n, pairs, 2)))
    sc = None
    if scaling is not None:
        sc = ctypes.byref(_RopeScaling(ROPE_KIND[scaling.kind], scaling.factor,
                                       scaling.original_len, scaling.low, scaling.high,
                                       scaling.amplitude))
    st = load_library().kvq_rope_table(table.data_ptr(), n, 2 * pairs, float(base), sc,
                                       _raw_stream(dev, stream))
    _check(st, "kvq_rope_table")
    return table


@dataclass
class Rope:
    """A layer's norm and rotation: table of kvq_rope_table (None: no rotation), pairs
    (2i, 2i+1) if interleaved else (i, i + rot_dim/2), and the norms' weights (bf16
    [head_dim], None: no norm)."""
    table: Optional[torch.Tensor]
    interleaved: bool = False
    q_weight: Optional[torch.Tensor] = None
    k_weight: Optional[torch.Tensor] = None
    eps: float = 1e-6
    weight_offset: float = 0.0

    def desc(self, head_dim: int, dev: int) -> _RopeDesc:
        rot, count, table = 0, 0, self.table
        if table is not None:
            _need(table.dim() == 3, "table must have shape (positions, rot_dim / 2, 2)")
            count, pairs = table.shape[:2]
            rot = 2 * pairs
            _tensors(dev, ("table", table, torch.float32, (count, pairs, 2)))
        for name, w in (("q_weight", self.q_weight), ("k_weight", self.k_weight)):
            if w is not None:
                _tensors(dev, (name, w, torch.bfloat16, (head_dim,)))
        return _RopeDesc(head_dim, rot, self.interleaved, self.eps, self.weight_offset,
                         _address(self.q_weight), _address(self.k_weight), _address(table), count)


def kvq_norm_rope(rope: Rope, query: torch.Tensor, key: torch.Tensor, positions: torch.Tensor,
                  query_out: torch.Tensor, key_out: torch.Tensor, stream=None) -> None:
    """query_out, key_out <- normalised and rotated query [T, Hq, D] and key [T, Hkv, D]
    (bf16, token strides free; an output may be its own input)."""
    t, hq, d = query.shape
    q, kv = (t, hq, d), (t, key.shape[1], d)
    dev = _device_of("query", query)
    qs, ks = _rows(dev, "query", query, q), _rows(dev, "key", key, kv)
    qos, kos = _rows(dev, "query_out", query_out, q), _rows(dev, "key_out", key_out, kv)
    _tensors(dev, ("positions", positions, torch.int32, (t,)))
    r = rope.desc(d, dev)
    st = load_library().kvq_norm_rope(ctypes.byref(r), query_out.data_ptr(), qos, key_out.data_ptr(),
                                      kos, query.data_ptr(), qs, key.data_ptr(), ks,
                                      positions.data_ptr(), t, hq, kv[1],
                                      _raw_stream(dev, stream))
    _check(st, "kvq_norm_rope")


def kvq_norm_rope_write(rope: Rope, cache: KVCache, query: torch.Tensor, key: torch.Tensor,
                        value: torch.Tensor, positions: torch.Tensor, slot_mapping: torch.Tensor,
                        query_out: torch.Tensor, stream=None) -> torch.Tensor:
    """kvq_norm_rope of the queries into query_out, and of the keys straight into the
    cache, together with the values, at slot_mapping (int64 [T])."""
    t, hq, _ = query.shape
    d = cache.head_dim
    q, kv = (t, hq, d), (t, cache.num_kv_heads, d)
    dev = _device_of("query", query)
    qs, qos = _rows(dev, "query", query, q), _rows(dev, "query_out", query_out, q)
    ks, vs = _rows(dev, "key", key, kv), _rows(dev, "value", value, kv)
    _tensors(dev, ("positions", positions, torch.int32, (t,)),
             ("slot_mapping", slot_mapping, torch.int64, (t,)))
    r, c = rope.desc(d, dev), _cache_desc(dev, cache)
    st = load_library().kvq_norm_rope_write(
        ctypes.byref(r), ctypes.byref(c), cache.k_cache.data_ptr(), cache.v_cache.data_ptr(),
        query_out.data_ptr(), qos, query.data_ptr(), qs, key.data_ptr(), ks, value.data_ptr(), vs,
        positions.data_ptr(), slot_mapping.data_ptr(), t, hq, _raw_stream(dev, stream))
    _check(st, "kvq_norm_rope_write")
    return query_out


def kvq_decode_window(cache: KVCache, query: torch.Tensor, out: torch.Tensor,
                      block_table: torch.Tensor, context_lens: torch.Tensor, max_context_len: int,
                      sm_scale: float, window: int, num_sinks: int = 0,
                      workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                      new_key: Optional[torch.Tensor] = None,
                      new_value: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """kvq_paged_decode (or, with new_key / new_value, kvq_decode_append) of queries that
    see the last `window` tokens of their context and its first num_sinks."""
    s, hq, _ = query.shape
    rows, width = (s, hq, cache.head_dim), block_table.shape[-1]
    _int32(max_context_len=max_context_len, window=window, num_sinks=num_sinks, num_ctas=num_ctas)
    dev = _device_of("query", query)
    _tensors(dev, ("query", query, torch.bfloat16, rows), ("out", out, torch.bfloat16, rows),
             ("block_table", block_table, torch.int32, (s, width)),
             ("context_lens", context_lens, torch.int32, (s,)))
    _need((new_key is None) == (new_value is None), "new_key and new_value come together")
    ks = vs = 0
    if new_key is not None:
        kv = (s, cache.num_kv_heads, cache.head_dim)
        ks, vs = _rows(dev, "new_key", new_key, kv), _rows(dev, "new_value", new_value, kv)
    c = _cache_desc(dev, cache)
    st = load_library().kvq_decode_window(
        ctypes.byref(c), cache.k_cache.data_ptr(), cache.v_cache.data_ptr(), _address(new_key),
        _address(new_value), ks, vs, out.data_ptr(), query.data_ptr(), s, hq, block_table.data_ptr(),
        width, context_lens.data_ptr(), max_context_len, float(sm_scale), window, num_sinks, num_ctas,
        _address(workspace), _workspace(dev, workspace), _raw_stream(dev, stream))
    _check(st, "kvq_decode_window")
    return out


def kvq_prefill_workspace_size(cache: KVCache, num_seqs: int, num_q_heads: int, total_q: int,
                               max_query_len: int, max_context_len: int) -> int:
    _int32(num_seqs=num_seqs, num_q_heads=num_q_heads, max_query_len=max_query_len, max_context_len=max_context_len)
    n = ctypes.c_size_t(0)
    c = cache.desc()
    _check(load_library().kvq_prefill_workspace_size(ctypes.byref(c), num_seqs, num_q_heads,
                                                     total_q, max_query_len, max_context_len,
                                                     ctypes.byref(n)), "kvq_prefill_workspace_size")
    return int(n.value)


def kvq_paged_prefill(cache: KVCache, query: torch.Tensor, out: torch.Tensor,
                      cu_query: torch.Tensor, block_table: torch.Tensor,
                      context_lens: torch.Tensor, max_query_len: int, max_context_len: int,
                      sm_scale: float, window: int = 0, num_sinks: int = 0,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out <- attention of each sequence's new tokens (query: bf16 [total, Hq, D], packed;
    rows cu_query[s]..cu_query[s+1]-1 are sequence s's last positions) to its cached context
    of context_lens[s] tokens, causal, through `window` (0: no limit) and num_sinks."""
    s = context_lens.numel()
    n, hq, _ = query.shape
    rows, width = (n, hq, cache.head_dim), block_table.shape[-1]
    _int32(max_query_len=max_query_len, max_context_len=max_context_len, window=window, num_sinks=num_sinks)
    dev = _device_of("query", query)
    _tensors(dev, ("query", query, torch.bfloat16, rows), ("out", out, torch.bfloat16, rows),
             ("cu_query", cu_query, torch.int32, (s + 1,)),
             ("block_table", block_table, torch.int32, (s, width)),
             ("context_lens", context_lens, torch.int32, (s,)))
    c = _cache_desc(dev, cache)
    st = load_library().kvq_paged_prefill(
        ctypes.byref(c), cache.k_cache.data_ptr(), cache.v_cache.data_ptr(), out.data_ptr(),
        query.data_ptr(), cu_query.data_ptr(), s, n, max_query_len, hq, block_table.data_ptr(), width,
        context_lens.data_ptr(), max_context_len, float(sm_scale), window, num_sinks,
        _address(workspace), _workspace(dev, workspace), _raw_stream(dev, stream))
    _check(st, "kvq_paged_prefill")
    return out


def kvq_hadamard(x: torch.Tensor, signs: Optional[torch.Tensor] = None, inverse: bool = False,
                 stream=None) -> torch.Tensor:
    """In-place rotation of the rows of x (float32 or bf16, [..., D], contiguous)."""
    lib = load_library()
    assert x.is_contiguous()
    dt = {torch.float32: 0, torch.bfloat16: 1}[x.dtype]
    dim = x.shape[-1]
    rows = x.numel() // dim if dim else 0
    st = lib.kvq_hadamard(_ptr(x), dt, rows, dim, _ptr(signs), int(inverse), _stream(stream))
    _check(st, "kvq_hadamard")
    return x


def kvq_calibrate_scale(x: torch.Tensor, qmax: float, out: torch.Tensor, stream=None):
    """out (device float32 [1]) <- absmax(x) / qmax (1.0 for an all-zero x)."""
    lib = load_library()
    assert x.dtype == torch.bfloat16 and x.is_contiguous() and out.dtype == torch.float32
    st = lib.kvq_calibrate_scale(_ptr(x), x.numel(), float(qmax), _ptr(out), _stream(stream))
    _check(st, "kvq_calibrate_scale")
    return out


def kvq_calibrate_head_scales(x: torch.Tensor, qmax: float, out: torch.Tensor, stream=None):
    """out (device float32 [Hkv]) <- per-kv-head absmax of x [T, Hkv, D] / qmax."""
    lib = load_library()
    assert x.dtype == torch.bfloat16 and x.dim() == 3 and out.dtype == torch.float32
    assert x.stride(2) == 1 and x.stride(1) == x.shape[2] and out.numel() == x.shape[1]
    st = lib.kvq_calibrate_head_scales(_ptr(x), x.shape[0], x.shape[1], x.shape[2], x.stride(0),
                                       float(qmax), _ptr(out), _stream(stream))
    _check(st, "kvq_calibrate_head_scales")
    return out


def kvq_debug_arm_wait_timeout(polls: int, cta: int, tile: int) -> None:
    """Test hook: the next decode or chunk-attention launch polls each pipeline wait at
    most `polls` times, and CTA `cta` (first kv-head group; first part of the keys) never
    gets its range's tile `tile`, so that a wait runs out (KVQ_DEVERR_TIMEOUT); one
    launch only."""
    _check(load_library().kvq_debug_arm_wait_timeout(polls, cta, tile),
           "kvq_debug_arm_wait_timeout")


def kvq_get_device_error(stream=None) -> int:
    """Synchronize, then read-and-clear the device error word (KVQ_DEVERR_* bits)."""
    lib = load_library()
    bits = ctypes.c_uint32(0)
    _check(lib.kvq_get_device_error(_stream(stream), ctypes.byref(bits)), "kvq_get_device_error")
    return int(bits.value)


def kvq_version() -> str:
    return load_library().kvq_version().decode()
