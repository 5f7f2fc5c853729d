"""Python binding of libpa.so: the C ABI in include/pa.h, same names.

Argument marshalling only. Each call checks that its tensors are CUDA,
contiguous and of the expected dtype, passes their pointers and the current
torch stream to the C entry point, and raises PaError on a nonzero return.
Every step of the computation runs in the library's kernels. There is no
fallback: if libpa.so is missing, importing this module raises ImportError.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

PA_DTYPE_F32, PA_DTYPE_BF16 = 0, 1
BLOCK_SIZE = 16

PA_STATUS_BAD_BLOCK_ID = 0x1
PA_STATUS_BAD_SLOT = 0x2
PA_STATUS_BAD_CONTEXT = 0x4
PA_STATUS_WAIT_TIMEOUT = 0x8
PA_STATUS_BAD_QUERY = 0x10
PA_ABI_VERSION = 7


class PaShape(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("kv_fp8", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
    ]


class PaRopePlan(ctypes.Structure):
    """pa_rope_plan: what pa_rope_init makes and the rotary calls take."""
    _fields_ = [
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("mscale", ctypes.c_float),
        ("reserved", ctypes.c_int32),
        ("step", ctypes.c_uint64 * 64),
    ]


EXPORTED = [
    "pa_reshape_and_cache", "pa_decode_workspace_bytes", "pa_decode", "pa_decode_partials", "pa_decode_merge",
    "pa_prefill_chunk",
    "pa_get_status", "pa_strerror", "pa_last_cuda_error", "pa_abi_version", "pa_decode_noalloc",
    "pa_copy_blocks", "pa_swap_blocks",
    "pa_rope_init", "pa_rope", "pa_rope_and_cache", "pa_cache_block8", "pa_decode_block8_workspace_bytes",
    "pa_decode_block8", "pa_decode_weights_workspace_bytes", "pa_decode_weights", "pa_evict",
]

PA_KV_BLOCK_E4M3, PA_KV_BLOCK_INT8 = 2, 3
PA_ROPE_MAX_DIM = 128
_ROPE_SCALING = {"none": 0, "linear": 1, "base": 2, "parts": 3}

PA_ERR_SCRATCH_LIMIT = -7
PA_NOALLOC_SCRATCH_BYTES = 16 << 20


def _load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError("libpa.so not built at %s: run paged_kv_cache_366_b200/build.py" % path)
    lib = ctypes.CDLL(path)
    P, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    SP = ctypes.POINTER(PaShape)
    lib.pa_reshape_and_cache.argtypes = [P, P, P, P, P, I64, SP, P]
    lib.pa_reshape_and_cache.restype = ctypes.c_int
    lib.pa_decode_workspace_bytes.argtypes = [I32, I32, I32, SP]
    lib.pa_decode_workspace_bytes.restype = I64
    for name in ("pa_decode", "pa_decode_partials", "pa_decode_merge"):
        getattr(lib, name).argtypes = [P, P, P, P, P, I32, P, I32, I32, F, I32, P, I64, SP, P]
        getattr(lib, name).restype = ctypes.c_int
    lib.pa_prefill_chunk.argtypes = [P, P, P, P, P, I32, P, P, I32, I32, I32, F, SP, P]
    lib.pa_prefill_chunk.restype = ctypes.c_int
    lib.pa_decode_noalloc.argtypes = [P, P, P, P, P, I32, P, I32, I32, F, I32, SP, P]
    lib.pa_decode_noalloc.restype = ctypes.c_int
    lib.pa_copy_blocks.argtypes = [P, P, P, I64, SP, P]
    lib.pa_copy_blocks.restype = ctypes.c_int
    lib.pa_swap_blocks.argtypes = [P, P, P, I64, I64, I64, I64, P]
    lib.pa_swap_blocks.restype = ctypes.c_int
    RP, D = ctypes.POINTER(PaRopePlan), ctypes.c_double
    lib.pa_rope_init.argtypes = [RP, I32, I32, D, I32, D, D, D, D, D]
    lib.pa_rope.argtypes = [P, P, P, P, I64, I64, P, I64, RP, SP, P]
    lib.pa_rope_and_cache.argtypes = [P, P, P, P, I64, I64, I64, P, P, P, P, I64, RP, SP, P]
    lib.pa_cache_block8.argtypes = [P, P, P, P, P, P, P, I64, SP, P]
    lib.pa_decode_block8.argtypes = [P, P, P, P, P, P, P, I32, P, I32, I32, F, I32, P, I64, SP, P]
    lib.pa_decode_weights.argtypes = [P, P, I32, P, P, P, P, P, P, I32, P, I32, I32, F, I32, P, I64, SP, P]
    lib.pa_evict.argtypes = [P, P, P, P, P, I32, P, I32, P, P, I32, P, P, P, I32, I32, I32, I32, I32, SP, P]
    for name in ("pa_rope_init", "pa_rope", "pa_rope_and_cache", "pa_cache_block8", "pa_decode_block8",
                 "pa_decode_weights", "pa_evict"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("pa_decode_block8_workspace_bytes", "pa_decode_weights_workspace_bytes"):
        getattr(lib, name).argtypes = [I32, I32, I32, SP]
        getattr(lib, name).restype = I64
    lib.pa_get_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), P]
    lib.pa_get_status.restype = ctypes.c_int
    lib.pa_strerror.argtypes = [ctypes.c_int]
    lib.pa_strerror.restype = ctypes.c_char_p
    lib.pa_last_cuda_error.argtypes = []
    lib.pa_last_cuda_error.restype = ctypes.c_int
    lib.pa_abi_version.argtypes = []
    lib.pa_abi_version.restype = ctypes.c_int
    return lib


lib = _load()
if lib.pa_abi_version() != PA_ABI_VERSION:
    raise ImportError("libpa.so has ABI version %d, the binding expects %d: rebuild it"
                      % (lib.pa_abi_version(), PA_ABI_VERSION))


class PaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        msg = "%s: %s (%d)" % (fn, lib.pa_strerror(code).decode(), code)
        if code == -5:
            msg += ", cudaError %d" % lib.pa_last_cuda_error()
        super().__init__(msg)


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise PaError(fn, rc)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return PA_DTYPE_BF16
    if dt == torch.float32:
        return PA_DTYPE_F32
    raise ValueError("dtype must be bfloat16 or float32, got %s" % dt)


def shape_of(k_cache: torch.Tensor, num_heads: int, k_scale: float = 0.0, v_scale: float = 0.0) -> PaShape:
    """pa_shape of a pool [NB, 16, Hk, D] read by `num_heads` query heads.

    A uint8 pool holds FP8 E4M3 codes (values code * k_scale / code * v_scale)
    next to bf16 q/out and new tokens.
    """
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_blocks, block_size, num_kv_heads, head_dim]")
    nb, bs, hk, d = k_cache.shape
    fp8 = k_cache.dtype == torch.uint8
    return PaShape(num_heads=int(num_heads), num_kv_heads=int(hk), head_dim=int(d), block_size=int(bs),
                   num_blocks=int(nb), dtype=PA_DTYPE_BF16 if fp8 else _dtype_code(k_cache.dtype),
                   kv_fp8=1 if fp8 else 0, k_scale=float(k_scale), v_scale=float(v_scale))


def _same_dtype_kv(q_like, caches):
    """q/out/new tokens share one dtype; caches share it or are uint8 FP8 codes with bf16 elsewhere."""
    _same_dtype(*q_like)
    _same_dtype(*caches)
    if caches[0].dtype == torch.uint8:
        if q_like[0].dtype != torch.bfloat16:
            raise ValueError("an FP8 cache goes with bf16 q, out and new tokens")
    elif caches[0].dtype != q_like[0].dtype:
        raise ValueError("q/out/k/v and the caches must share one dtype")


def _same_dtype(*ts):
    dts = {t.dtype for t in ts}
    if len(dts) != 1:
        raise ValueError("q/k/v/caches/out must share one dtype, got %s" % sorted(map(str, dts)))


def _int(t: torch.Tensor, dt: torch.dtype, name: str):
    if t.dtype != dt:
        raise ValueError("%s must be %s" % (name, dt))


def pa_reshape_and_cache(k, v, k_cache, v_cache, slot_mapping, stream=None, k_scale: float = 0.0,
                         v_scale: float = 0.0) -> None:
    """Write each new token's K/V row into its slot of the pool (bit-exact copy, or FP8 quantization)."""
    _same_dtype_kv((k, v), (k_cache, v_cache))
    _int(slot_mapping, torch.int64, "slot_mapping")
    shape = shape_of(k_cache, k_cache.shape[2], k_scale, v_scale)
    if k.shape[1:] != k_cache.shape[2:] or v.shape != k.shape or slot_mapping.shape[0] != k.shape[0]:
        raise ValueError("k, v must be [T, Hk, D] matching the cache; slot_mapping [T]")
    _check("pa_reshape_and_cache",
           lib.pa_reshape_and_cache(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
                                    k.shape[0], ctypes.byref(shape), _stream(stream)))


def pa_decode_workspace_bytes(num_seqs: int, max_context_len: int, partition_tokens: int, shape: PaShape) -> int:
    n = lib.pa_decode_workspace_bytes(int(num_seqs), int(max_context_len), int(partition_tokens),
                                      ctypes.byref(shape))
    if n < 0:
        raise PaError("pa_decode_workspace_bytes", int(n))
    return int(n)


def _decode(fn: str, out, q, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
            partition_tokens, workspace, stream, k_scale, v_scale) -> None:
    _same_dtype_kv((out, q), (k_cache, v_cache))
    _int(block_tables, torch.int32, "block_tables")
    _int(context_lens, torch.int32, "context_lens")
    B, H, D = q.shape
    if out.shape != q.shape or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("q, out [B, H, D]; block_tables [B, MB]; context_lens [B]")
    shape = shape_of(k_cache, H, k_scale, v_scale)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(fn,
           getattr(lib, fn)(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                            block_tables.shape[1], _ptr(context_lens), B, int(max_context_len), float(scale),
                            int(partition_tokens), _ptr(workspace), ws_bytes, ctypes.byref(shape),
                            _stream(stream)))


def pa_decode(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int, scale: float,
              partition_tokens: int = 0, workspace: Optional[torch.Tensor] = None, stream=None,
              k_scale: float = 0.0, v_scale: float = 0.0) -> None:
    """Decode attention of one query token per sequence over its paged context."""
    _decode("pa_decode", out, q, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
            partition_tokens, workspace, stream, k_scale, v_scale)


def pa_decode_partials(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int, scale: float,
                       partition_tokens: int = 0, workspace: Optional[torch.Tensor] = None, stream=None,
                       k_scale: float = 0.0, v_scale: float = 0.0) -> None:
    """The first of pa_decode's two launches: the partition pass (arguments as pa_decode)."""
    _decode("pa_decode_partials", out, q, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
            partition_tokens, workspace, stream, k_scale, v_scale)


def pa_decode_merge(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int, scale: float,
                    partition_tokens: int = 0, workspace: Optional[torch.Tensor] = None, stream=None,
                    k_scale: float = 0.0, v_scale: float = 0.0) -> None:
    """The second of pa_decode's two launches: the merge of cut units (arguments as pa_decode)."""
    _decode("pa_decode_merge", out, q, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
            partition_tokens, workspace, stream, k_scale, v_scale)


def pa_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int, scale: float,
                      partition_tokens: int = 0, stream=None, k_scale: float = 0.0, v_scale: float = 0.0) -> None:
    """pa_decode without a workspace argument, for callers that cannot allocate device memory.

    The split-context partials go to a PA_NOALLOC_SCRATCH_BYTES array built
    into the library (held on every device that loads it). Requests that need
    more raise PaError with PA_ERR_SCRATCH_LIMIT. Calls that may overlap on
    one GPU share that array and must not run concurrently. Make the first
    call on each device outside stream capture. A uint8 (FP8 E4M3) pool takes
    k_scale and v_scale as in pa_decode.
    """
    _same_dtype_kv((out, q), (k_cache, v_cache))
    _int(block_tables, torch.int32, "block_tables")
    _int(context_lens, torch.int32, "context_lens")
    B, H, D = q.shape
    if out.shape != q.shape or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("q, out [B, H, D]; block_tables [B, MB]; context_lens [B]")
    shape = shape_of(k_cache, H, k_scale, v_scale)
    _check("pa_decode_noalloc",
           lib.pa_decode_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                 block_tables.shape[1], _ptr(context_lens), B, int(max_context_len), float(scale),
                                 int(partition_tokens), ctypes.byref(shape), _stream(stream)))


def pa_prefill_chunk(out, q, k_cache, v_cache, block_tables, cu_q_lens, context_lens, max_q_len: int,
                     scale: float, stream=None, k_scale: float = 0.0, v_scale: float = 0.0) -> None:
    """Causal attention of query chunks at their context offsets (bf16 q/out, D=128; bf16 caches, or uint8
    FP8 E4M3 caches with their k_scale / v_scale)."""
    _same_dtype_kv((out, q), (k_cache, v_cache))
    _int(block_tables, torch.int32, "block_tables")
    _int(cu_q_lens, torch.int32, "cu_q_lens")
    _int(context_lens, torch.int32, "context_lens")
    T, H, D = q.shape
    B = context_lens.shape[0]
    if out.shape != q.shape or block_tables.shape[0] != B or cu_q_lens.shape[0] != B + 1:
        raise ValueError("q, out [T, H, D]; block_tables [B, MB]; cu_q_lens [B+1]; context_lens [B]")
    shape = shape_of(k_cache, H, k_scale, v_scale)
    _check("pa_prefill_chunk",
           lib.pa_prefill_chunk(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                block_tables.shape[1], _ptr(cu_q_lens), _ptr(context_lens), B, int(max_q_len), T,
                                float(scale), ctypes.byref(shape), _stream(stream)))


def pa_copy_blocks(k_cache, v_cache, block_pairs, stream=None) -> None:
    """Copy whole blocks inside the pool: block_pairs int64 [n, 2] of (src, dst), on the device.

    A block8 pool's codes are copied as bytes; its scales' rows (k_scales[dst] = k_scales[src]) are the caller's.
    """
    _same_dtype(k_cache, v_cache)
    if k_cache.dtype == torch.int8:
        k_cache, v_cache = k_cache.view(torch.uint8), v_cache.view(torch.uint8)
    _int(block_pairs, torch.int64, "block_pairs")
    shape = shape_of(k_cache, k_cache.shape[2], 1.0, 1.0)
    _check("pa_copy_blocks", lib.pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_pairs),
                                                block_pairs.numel() // 2, ctypes.byref(shape), _stream(stream)))


def _any_ptr(t: torch.Tensor):
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    if not t.is_cuda and not t.is_pinned():
        raise ValueError("host tensors must be pinned")
    return ctypes.c_void_p(t.data_ptr())


def pa_swap_blocks(dst, src, block_pairs, stream=None) -> None:
    """Copy blocks of one pool between device and pinned host memory: block_pairs int64 [n, 2] of (src, dst)."""
    if dst.dtype != src.dtype or dst.shape[1:] != src.shape[1:]:
        raise ValueError("dst and src pools must have the same dtype and block shape")
    _int(block_pairs, torch.int64, "block_pairs")
    bb = src[0].numel() * src.element_size()
    _check("pa_swap_blocks", lib.pa_swap_blocks(_any_ptr(dst), _any_ptr(src), _any_ptr(block_pairs),
                                                block_pairs.numel() // 2, src.shape[0], dst.shape[0], bb,
                                                _stream(stream)))


# ---- rotary positions, the block-scaled 8-bit cache, weight-counting decode, eviction ----
#
# These are called once a layer and step, some for kernels of a few microseconds, so the checks are kept short:
# plain comparisons, data_ptr() as an int, the current stream's handle without a Stream object, and pa_shape structs
# shared by their values.


@functools.lru_cache(maxsize=256)
def _shape(num_heads, num_kv_heads, head_dim, block_size, num_blocks, dtype, kv_fp8, k_scale=0.0, v_scale=0.0):
    return PaShape(num_heads=num_heads, num_kv_heads=num_kv_heads, head_dim=head_dim, block_size=block_size,
                   num_blocks=num_blocks, dtype=dtype, kv_fp8=kv_fp8, k_scale=k_scale, v_scale=v_scale)


def _device_of(tensors) -> int:
    """The one device of the tensors, which is the current one; all are contiguous (None entries are skipped)."""
    dev = tensors[0].get_device()
    if dev < 0:
        raise ValueError("tensor must be on a CUDA device")
    for t in tensors:
        if t is not None:
            if t.get_device() != dev:
                raise ValueError("all tensors must be on one CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensor must be contiguous")
    if dev != _current_device():
        raise ValueError("tensors are on cuda:%d, which is not the current device" % dev)
    return dev


def _current_device() -> int:
    # a CUDA tensor exists, so the runtime is up: the plain query, without torch.cuda's initialisation check
    return torch._C._cuda_getDevice()


def _stream_on(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError("the stream and the tensors are on different devices")
    return stream.cuda_stream


def _optional(t):
    return t.data_ptr() if t is not None else None


def pa_rope_init(rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, low: float = 1.0, high: float = 32.0, original_len: float = 0.0,
                 mscale: float = 1.0) -> PaRopePlan:
    """Plan of a rotary embedding of the first rot_dim dims. scaling: none, linear, base or parts."""
    if scaling not in _ROPE_SCALING:
        raise ValueError("scaling must be one of %s, got %r" % (sorted(_ROPE_SCALING), scaling))
    plan = PaRopePlan()
    _check("pa_rope_init", lib.pa_rope_init(ctypes.byref(plan), int(rot_dim), 1 if interleaved else 0, float(base),
                                            _ROPE_SCALING[scaling], float(factor), float(low), float(high),
                                            float(original_len), float(mscale)))
    return plan


def _row_stride(t: torch.Tensor, dev: int, heads: int, dim: int) -> int:
    """Token stride (elements) of [T, heads, dim] rows whose last two dims are contiguous."""
    if t.get_device() != dev:
        raise ValueError("all tensors must be on one CUDA device")
    stride = t.stride()
    if stride[2] != 1 or (stride[1] != dim and heads > 1):
        raise ValueError("q, k and v rows must have contiguous heads (any token stride)")
    return stride[0] if t.shape[0] > 1 else heads * dim


def pa_rope(q_out, k_out, q, k, positions, plan: PaRopePlan, stream=None) -> None:
    """Rotate q [T, H, D] and k [T, Hk, D] by position (token strides are free; in place where contiguous)."""
    dt = q.dtype
    if k.dtype != dt or q_out.dtype != dt or k_out.dtype != dt:
        raise ValueError("q, k and their outputs must share one dtype")
    _int(positions, torch.int64, "positions")
    T, H, D = q.shape
    Hk = k.shape[1]
    if q_out.shape != q.shape or k.shape != (T, Hk, D) or k_out.shape != k.shape or positions.shape != (T,):
        raise ValueError("q, q_out [T, H, D]; k, k_out [T, Hk, D]; positions [T]")
    dev = _device_of((q_out, k_out, positions))
    shape = _shape(H, Hk, D, BLOCK_SIZE, 1, _dtype_code(dt), 0)
    _check("pa_rope", lib.pa_rope(q_out.data_ptr(), k_out.data_ptr(), q.data_ptr(), k.data_ptr(),
                                  _row_stride(q, dev, H, D), _row_stride(k, dev, Hk, D), positions.data_ptr(), T,
                                  plan, shape, _stream_on(stream, dev)))


def pa_rope_and_cache(q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, plan: PaRopePlan, stream=None,
                      k_scale: float = 0.0, v_scale: float = 0.0) -> None:
    """Rotate q [T, H, D] into q_out, and write the rotated k and v [T, Hk, D] to their slots of the pool."""
    dt = q.dtype
    if q_out.dtype != dt or k.dtype != dt or v.dtype != dt:
        raise ValueError("q, q_out, k and v must share one dtype")
    _int(slot_mapping, torch.int64, "slot_mapping")
    _int(positions, torch.int64, "positions")
    T, H, D = q.shape
    shape = _pool_shape(k_cache, v_cache, H, D, dt, k_scale, v_scale, None, None)
    Hk = shape.num_kv_heads
    rows = (T, Hk, D)
    if (q_out.shape != q.shape or k.shape != rows or v.shape != rows or positions.shape != (T,)
            or slot_mapping.shape != (T,)):
        raise ValueError("q, q_out [T, H, D]; k, v [T, Hk, D]; slot_mapping, positions [T]")
    dev = _device_of((q_out, k_cache, v_cache, slot_mapping, positions))
    _check("pa_rope_and_cache",
           lib.pa_rope_and_cache(q_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                 _row_stride(q, dev, H, D), _row_stride(k, dev, Hk, D), _row_stride(v, dev, Hk, D),
                                 k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(),
                                 positions.data_ptr(), T, plan, shape, _stream_on(stream, dev)))


def shape_of_block8(k_codes: torch.Tensor, num_heads: int) -> PaShape:
    """pa_shape of a block8 pool [NB, 16, Hk, D]: uint8 E4M3 codes or int8 codes, beside bf16 q and out."""
    return PaShape.from_buffer_copy(_codes_shape(k_codes, num_heads))


def _codes_shape(k_codes: torch.Tensor, num_heads: int) -> PaShape:
    if k_codes.dim() != 4:
        raise ValueError("codes must be [num_blocks, block_size, num_kv_heads, head_dim]")
    dt = k_codes.dtype
    if dt != torch.uint8 and dt != torch.int8:
        raise ValueError("block8 codes are uint8 (E4M3) or int8, got %s" % dt)
    nb, bs, hk, d = k_codes.shape
    return _shape(int(num_heads), hk, d, bs, nb, PA_DTYPE_BF16,
                  PA_KV_BLOCK_E4M3 if dt == torch.uint8 else PA_KV_BLOCK_INT8)


def _block8_shape(k_codes, v_codes, k_scales, v_scales, num_heads) -> PaShape:
    shape = _codes_shape(k_codes, num_heads)
    if v_codes.dtype != k_codes.dtype or v_codes.shape != k_codes.shape:
        raise ValueError("k_codes and v_codes must have one shape and dtype")
    want = (shape.num_blocks, shape.num_kv_heads)
    if (k_scales.dtype != torch.float32 or v_scales.dtype != torch.float32 or k_scales.shape != want
            or v_scales.shape != want):
        raise ValueError("scales must be float32 [num_blocks, num_kv_heads]")
    return shape


def _pool_shape(k_cache, v_cache, num_heads, head_dim, dtype, k_scale, v_scale, k_scales, v_scales) -> PaShape:
    """The shape of a pool read or written next to q of `dtype`: a block8 pool where its scales are given."""
    if k_scales is not None or v_scales is not None:
        if k_scales is None or v_scales is None:
            raise ValueError("give both k_scales and v_scales, or neither")
        shape = _block8_shape(k_cache, v_cache, k_scales, v_scales, num_heads)
        fp8 = True
    else:
        if k_cache.dim() != 4:
            raise ValueError("k_cache must be [num_blocks, block_size, num_kv_heads, head_dim]")
        if v_cache.dtype != k_cache.dtype or v_cache.shape != k_cache.shape:
            raise ValueError("k_cache and v_cache must have one shape and dtype")
        nb, bs, hk, d = k_cache.shape
        fp8 = k_cache.dtype == torch.uint8
        shape = _shape(int(num_heads), hk, d, bs, nb, PA_DTYPE_BF16 if fp8 else _dtype_code(k_cache.dtype),
                       1 if fp8 else 0, float(k_scale), float(v_scale))
    if dtype != (torch.bfloat16 if fp8 else k_cache.dtype):
        raise ValueError("q, out and new tokens must have the pool's dtype (bf16 beside 8-bit pools)")
    if shape.head_dim != head_dim:
        raise ValueError("q and the pool must have one head_dim")
    return shape


def pa_cache_block8(k, v, k_codes, v_codes, k_scales, v_scales, slot_mapping, stream=None) -> None:
    """Append new tokens' bf16 K/V rows to a block8 pool; the tokens of one block are neighbours in the call."""
    shape = _block8_shape(k_codes, v_codes, k_scales, v_scales, k_codes.shape[2])
    _int(k, torch.bfloat16, "k")
    _int(v, torch.bfloat16, "v")
    _int(slot_mapping, torch.int64, "slot_mapping")
    T = k.shape[0]
    rows = (T, shape.num_kv_heads, shape.head_dim)
    if k.shape != rows or v.shape != rows or slot_mapping.shape != (T,):
        raise ValueError("k, v must be [T, Hk, D] matching the pool; slot_mapping [T]")
    dev = _device_of((k, v, k_codes, v_codes, k_scales, v_scales, slot_mapping))
    _check("pa_cache_block8",
           lib.pa_cache_block8(k.data_ptr(), v.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
                               k_scales.data_ptr(), v_scales.data_ptr(), slot_mapping.data_ptr(), T, shape,
                               _stream_on(stream, dev)))


def pa_decode_block8_workspace_bytes(num_seqs: int, max_context_len: int, partition_tokens: int,
                                     shape: PaShape) -> int:
    n = lib.pa_decode_block8_workspace_bytes(int(num_seqs), int(max_context_len), int(partition_tokens), shape)
    if n < 0:
        raise PaError("pa_decode_block8_workspace_bytes", int(n))
    return int(n)


def _check_decode(out, q, block_tables, context_lens):
    _int(block_tables, torch.int32, "block_tables")
    _int(context_lens, torch.int32, "context_lens")
    B = q.shape[0]
    if (out.dtype != q.dtype or q.dim() != 3 or out.shape != q.shape or block_tables.dim() != 2
            or block_tables.shape[0] != B or context_lens.shape != (B,)):
        raise ValueError("q, out [B, H, D] of one dtype; block_tables [B, MB]; context_lens [B]")


def pa_decode_block8(out, q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, max_context_len: int,
                     scale: float, partition_tokens: int = 0, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """pa_decode over a block8 pool: uint8 (E4M3) or int8 codes with fp32 scales [NB, Hk]."""
    _check_decode(out, q, block_tables, context_lens)
    B, H, D = q.shape
    shape = _pool_shape(k_codes, v_codes, H, D, q.dtype, 0.0, 0.0, k_scales, v_scales)
    dev = _device_of((out, q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, workspace))
    _check("pa_decode_block8",
           lib.pa_decode_block8(out.data_ptr(), q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
                                k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(),
                                block_tables.shape[1], context_lens.data_ptr(), B, int(max_context_len), float(scale),
                                int(partition_tokens), _optional(workspace),
                                workspace.nbytes if workspace is not None else 0, shape, _stream_on(stream, dev)))


def pa_decode_weights_workspace_bytes(num_seqs: int, max_context_len: int, partition_tokens: int,
                                      shape: PaShape) -> int:
    n = lib.pa_decode_weights_workspace_bytes(int(num_seqs), int(max_context_len), int(partition_tokens), shape)
    if n < 0:
        raise PaError("pa_decode_weights_workspace_bytes", int(n))
    return int(n)


def pa_decode_weights(out, weights, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
                      scale: float, partition_tokens: int = 0, workspace: Optional[torch.Tensor] = None, stream=None,
                      k_scale: float = 0.0, v_scale: float = 0.0, k_scales: Optional[torch.Tensor] = None,
                      v_scales: Optional[torch.Tensor] = None) -> None:
    """Decode that also adds each entry's attention weight to weights [B, Hk, W] (float32, W >= max_context_len).

    A pool with k_scales and v_scales [NB, Hk] is a block8 pool; a uint8 pool without them takes k_scale, v_scale.
    """
    _check_decode(out, q, block_tables, context_lens)
    _int(weights, torch.float32, "weights")
    B, H, D = q.shape
    shape = _pool_shape(k_cache, v_cache, H, D, q.dtype, k_scale, v_scale, k_scales, v_scales)
    if weights.dim() != 3 or weights.shape[0] != B or weights.shape[1] != shape.num_kv_heads:
        raise ValueError("weights must be [B, Hk, W]")
    dev = _device_of((out, weights, q, k_cache, v_cache, block_tables, context_lens, workspace, k_scales, v_scales))
    _check("pa_decode_weights",
           lib.pa_decode_weights(out.data_ptr(), weights.data_ptr(), weights.shape[2], q.data_ptr(),
                                 k_cache.data_ptr(), v_cache.data_ptr(), _optional(k_scales), _optional(v_scales),
                                 block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), B,
                                 int(max_context_len), float(scale), int(partition_tokens), _optional(workspace),
                                 workspace.nbytes if workspace is not None else 0, shape, _stream_on(stream, dev)))


def pa_evict(k_cache, v_cache, weights, block_tables, context_lens, dst_block_tables, new_weights, new_context_lens,
             kept, sinks: int, recent: int, max_context_len: int, stream=None,
             k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None) -> None:
    """Cut every sequence's cache to kept.shape[2] entries for each KV head, copied into dst_block_tables' blocks.

    kept int32 [B, Hk, keep], new_weights float32 [B, Hk, 16 * dst_block_tables.shape[1]] and new_context_lens
    int32 [B] are written; the old blocks, tables, lengths and weights are only read.
    """
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_blocks, block_size, num_kv_heads, head_dim]")
    plain = k_scales is None and k_cache.dtype != torch.uint8
    shape = _pool_shape(k_cache, v_cache, k_cache.shape[2], k_cache.shape[3],
                        k_cache.dtype if plain else torch.bfloat16, 1.0, 1.0, k_scales, v_scales)
    for t, name in ((block_tables, "block_tables"), (context_lens, "context_lens"),
                    (dst_block_tables, "dst_block_tables"), (new_context_lens, "new_context_lens"), (kept, "kept")):
        _int(t, torch.int32, name)
    _int(weights, torch.float32, "weights")
    _int(new_weights, torch.float32, "new_weights")
    B, Hk = context_lens.shape[0], shape.num_kv_heads
    if (context_lens.shape != (B,) or new_context_lens.shape != (B,) or block_tables.dim() != 2
            or dst_block_tables.dim() != 2 or block_tables.shape[0] != B or dst_block_tables.shape[0] != B
            or kept.dim() != 3 or kept.shape[:2] != (B, Hk) or weights.dim() != 3 or weights.shape[:2] != (B, Hk)
            or new_weights.shape != (B, Hk, dst_block_tables.shape[1] * BLOCK_SIZE)):
        raise ValueError("context_lens, new_context_lens [B]; block_tables, dst_block_tables [B, .]; weights, kept "
                         "[B, Hk, .]; new_weights [B, Hk, 16 * dst blocks]")
    dev = _device_of((k_cache, v_cache, weights, block_tables, context_lens, dst_block_tables, new_weights,
                      new_context_lens, kept, k_scales, v_scales))
    _check("pa_evict",
           lib.pa_evict(k_cache.data_ptr(), v_cache.data_ptr(), _optional(k_scales), _optional(v_scales),
                        weights.data_ptr(), weights.shape[2], block_tables.data_ptr(), block_tables.shape[1],
                        context_lens.data_ptr(), dst_block_tables.data_ptr(), dst_block_tables.shape[1],
                        new_weights.data_ptr(), new_context_lens.data_ptr(), kept.data_ptr(), B,
                        int(max_context_len), kept.shape[2], int(sinks), int(recent), shape,
                        _stream_on(stream, dev)))


def pa_get_status(stream=None) -> int:
    """Synchronize the stream, return and clear the device status word (PA_STATUS_* flags)."""
    v = ctypes.c_uint32(0)
    _check("pa_get_status", lib.pa_get_status(ctypes.byref(v), _stream(stream)))
    return int(v.value)


def pa_strerror(code: int) -> str:
    return lib.pa_strerror(int(code)).decode()


def pa_abi_version() -> int:
    return int(lib.pa_abi_version())
