"""ctypes binding of libexl3.so (argument marshalling only).

Every function takes torch tensors that already live on the GPU, checks
dtype/contiguity/device, and passes raw pointers, sizes and the current CUDA
stream to the C ABI.  All arithmetic happens in the library's kernels.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libexl3.so")
_lib: Optional[ctypes.CDLL] = None

CODEBOOKS = {"3inst": 0, "mcg": 1, "mul1": 2}
_F16, _BF16 = 0, 1
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "split-k workspace too small", 4: "CUDA error"}


class _Heads(ctypes.Structure):  # exl3_heads_t
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Rope(ctypes.Structure):  # exl3_rope_t
    _fields_ = [("phases", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int), ("amplitude", ctypes.c_float)]


class _Cache(ctypes.Structure):  # exl3_kv_cache_t
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("format", ctypes.c_int)]


class _Norm(ctypes.Structure):  # exl3_head_norm_t
    _fields_ = [("weight", ctypes.c_void_p), ("head_stride", ctypes.c_int64), ("eps", ctypes.c_float)]


class _Axes(ctypes.Structure):  # exl3_rope_axes_t
    _fields_ = [("axes", ctypes.c_void_p), ("num_axes", ctypes.c_int32)]


class _Tables(ctypes.Structure):  # exl3_kv_tables_t
    _fields_ = [("block_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("held", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("table_width", ctypes.c_int32), ("page_size", ctypes.c_int32), ("capacity", ctypes.c_int32)]


class Exl3Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = ""
        if status == 4 and _lib is not None:
            detail = ": " + _lib.exl3_last_error().decode()
        super().__init__(f"{what} failed: {_STATUS.get(status, status)}{detail}")


def lib() -> ctypes.CDLL:
    """Load libexl3.so (built in-tree by ``build_ext.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (nvcc, sm_103a)"
        )
    L = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    L.exl3_input_transform.argtypes = [vp, ctypes.c_int, i64, i64, vp, i32, vp, vp]
    L.exl3_moe_input_transform.argtypes = [vp, ctypes.c_int, i64, i64, vp, i64, i32, vp, i32, vp, i32, i32, vp, vp]
    L.exl3_moe_input_transform.restype = ctypes.c_int
    L.exl3_moe_gemm.argtypes = [vp, i64, i64, vp, i32, ctypes.c_int, vp, vp, i32, vp, i32, i32, vp, ctypes.c_int,
                                i64, vp]
    L.exl3_moe_gemm.restype = ctypes.c_int
    L.exl3_moe_combine.argtypes = [vp, ctypes.c_int, i64, i64, vp, vp, i32, i32, vp, i64, i32, vp, vp, ctypes.c_int, vp]
    L.exl3_moe_combine.restype = ctypes.c_int
    L.exl3_input_transform_swiglu.argtypes = [vp, ctypes.c_int, i64, i64, vp, i32, vp, vp]
    L.exl3_input_transform_swiglu.restype = ctypes.c_int
    L.exl3_gemm.argtypes = [vp, i64, i64, vp, i32, ctypes.c_int, vp, vp, i32, vp, ctypes.c_int, i64, vp]
    L.exl3_gemm_splitk.argtypes = L.exl3_gemm.argtypes[:-1] + [vp, sz, vp]
    L.exl3_gemm_splitk_noalloc.argtypes = L.exl3_gemm.argtypes
    L.exl3_gemm_splitk_noalloc.restype = ctypes.c_int
    L.exl3_splitk_parts.argtypes = [i64, i64]
    L.exl3_splitk_parts.restype = i32
    L.exl3_splitk_workspace_bytes.argtypes = [i64, i64, i64]
    L.exl3_splitk_workspace_bytes.restype = sz
    L.exl3_test_gemm_shape.argtypes = [i32] + L.exl3_gemm.argtypes[:-1] + [vp, sz, vp]
    L.exl3_test_gemm_shape.restype = ctypes.c_int
    L.exl3_test_codebook.argtypes = [ctypes.c_int, vp, vp]
    L.exl3_test_unpack.argtypes = [vp, i32, ctypes.c_int, i64, i64, vp, vp]
    L.exl3_test_tile_plan.argtypes = [i64, i64, i64, ctypes.POINTER(ctypes.c_int32), i32, i32,
                                      ctypes.POINTER(ctypes.c_int64)]
    L.exl3_test_tile_plan.restype = ctypes.c_int
    L.exl3_test_wait_timeout.argtypes = [vp, vp]
    L.exl3_test_wait_timeout.restype = ctypes.c_int
    L.exl3_set_autotune.argtypes = [i32]
    L.exl3_set_autotune.restype = ctypes.c_int
    L.exl3_clear_autotune.argtypes = []
    L.exl3_clear_autotune.restype = ctypes.c_int
    L.exl3_autotune_entries.argtypes = []
    L.exl3_autotune_entries.restype = i64
    L.exl3_status_string.argtypes = [ctypes.c_int]
    L.exl3_status_string.restype = ctypes.c_char_p
    L.exl3_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    L.exl3_device_status.restype = ctypes.c_int
    L.exl3_last_error.argtypes = []
    L.exl3_last_error.restype = ctypes.c_char_p
    heads, cache, rope_p, f32 = ctypes.POINTER(_Heads), ctypes.POINTER(_Cache), ctypes.POINTER(_Rope), ctypes.c_float
    f64 = ctypes.c_double
    L.exl3_rope_phases.argtypes = [i32, f64, ctypes.c_int, f64, f64, f64, f64, vp, ctypes.POINTER(f32)]
    L.exl3_rope.argtypes = [heads, ctypes.c_int, i64, i32, i32, rope_p, vp, i64, i64, vp]
    L.exl3_kv_write.argtypes = [cache, heads, heads, ctypes.c_int, i64, vp, rope_p, heads, i32, vp, i64, i64, vp]
    L.exl3_kv_read.argtypes = [cache, vp, i64, ctypes.c_int, vp, vp, vp]
    L.exl3_attention_prompt.argtypes = [heads, heads, heads, ctypes.c_int, i64, i32, i32, i32, vp, i32, i32, f32, vp,
                                        i64, i64, vp]
    L.exl3_attention_paged_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32]
    L.exl3_attention_paged_workspace_bytes.restype = sz
    L.exl3_attention_paged.argtypes = [heads, ctypes.c_int, i64, i32, cache, vp, i32, vp, vp, i32, i32, i32, i32, f32,
                                       vp, i64, i64, vp, sz, vp]
    norm, axes, tables = ctypes.POINTER(_Norm), ctypes.POINTER(_Axes), ctypes.POINTER(_Tables)
    L.exl3_norm_rope.argtypes = [heads, ctypes.c_int, i64, i32, i32, norm, rope_p, axes, vp, i64, i64, vp]
    L.exl3_norm_kv_write.argtypes = [cache, heads, heads, ctypes.c_int, i64, vp, norm, norm, rope_p, axes, heads, i32, vp,
                                     i64, i64, vp]
    L.exl3_kv_plan.argtypes = [tables, vp, i64] + [vp] * 8
    L.exl3_kv_release.argtypes = [tables] + [vp] * 6
    L.exl3_attention_shared_workspace_bytes.argtypes = [i64] + [i32] * 5 + [ctypes.c_int] * 2 + [i32] * 3
    L.exl3_attention_shared_workspace_bytes.restype = sz
    L.exl3_attention_shared_pays.argtypes = [i64] + [i32] * 6 + [ctypes.c_int] * 2 + [i32] * 2
    L.exl3_attention_shared_pays.restype = ctypes.c_int
    L.exl3_attention_shared.argtypes = [heads, ctypes.c_int, i64, i32, cache, vp, i32, vp, vp, i32, vp, vp, i32, i32, i32,
                                        i32, f32, vp, i64, i64, vp, sz, vp]
    for name in ("exl3_norm_rope", "exl3_norm_kv_write", "exl3_kv_plan", "exl3_kv_release", "exl3_attention_shared"):
        getattr(L, name).restype = ctypes.c_int
    for name in ("exl3_rope_phases", "exl3_rope", "exl3_kv_write", "exl3_kv_read", "exl3_attention_prompt",
                 "exl3_attention_paged"):
        getattr(L, name).restype = ctypes.c_int
    for name in ("exl3_input_transform", "exl3_gemm", "exl3_gemm_splitk", "exl3_test_codebook", "exl3_test_unpack"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def device_status() -> int:
    """Read and clear the kernels' device-side error flags (synchronises the device)."""
    flags = ctypes.c_uint32(0)
    _check(lib().exl3_device_status(ctypes.byref(flags)), "exl3_device_status")
    return int(flags.value)


def test_wait_timeout(device="cuda") -> int:
    """exl3_test_wait_timeout: a kernel whose bounded wait gives up (about 2 s);
    returns the kernel's out word (0 when the wait gave up)."""
    out = torch.full((1,), 7, dtype=torch.int32, device=device)
    _check(lib().exl3_test_wait_timeout(_ptr(out), _stream(out)), "exl3_test_wait_timeout")
    return int(out.item())


def test_tile_plan(m: int, k: int, n: int, shard_cols: Sequence[int], split: bool = False) -> tuple:
    """The cost model's plan (host only): (shape, tail shape or -1, pair tiles, tail row, tail column)."""
    cols, ns = _cols(shard_cols)
    out = (ctypes.c_int64 * 5)()
    _check(lib().exl3_test_tile_plan(m, k, n, cols, ns, 1 if split else 0, out), "exl3_test_tile_plan")
    return tuple(int(v) for v in out)


def set_autotune(enable: bool) -> None:
    """Tile-shape autotune: time every shape on a key's first uncaptured call and keep the fastest."""
    _check(lib().exl3_set_autotune(1 if enable else 0), "exl3_set_autotune")


def clear_autotune() -> None:
    _check(lib().exl3_clear_autotune(), "exl3_clear_autotune")


def autotune_entries() -> int:
    return int(lib().exl3_autotune_entries())


def status_string(status: int) -> str:
    return lib().exl3_status_string(status).decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise Exl3Error(status, what)


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _cols(shard_cols: Sequence[int]):
    arr = (ctypes.c_int32 * len(shard_cols))(*[int(c) for c in shard_cols])
    return arr, len(shard_cols) - 1


def splitk_parts(k: int, n: int) -> int:
    return int(lib().exl3_splitk_parts(k, n))


def splitk_workspace_bytes(m: int, k: int, n: int) -> int:
    return int(lib().exl3_splitk_workspace_bytes(m, k, n))


def input_transform(x: torch.Tensor, suh: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """xh[s] = fp16(H(x * suh[s]) * 2^-4) for every shard; x bf16/fp16 [m, k], suh fp16 [S, k]."""
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("x must be bf16 or fp16")
    _need(x, x.dtype, "x")
    _need(suh, torch.float16, "suh")
    m, k = x.shape
    s = suh.shape[0]
    if out is None:
        out = torch.empty((s, m, k), dtype=torch.float16, device=x.device)
    _need(out, torch.float16, "out")
    st = lib().exl3_input_transform(_ptr(x), _BF16 if x.dtype == torch.bfloat16 else _F16, m, k, _ptr(suh), s,
                                    _ptr(out), _stream(x))
    _check(st, "exl3_input_transform")
    return out


def input_transform_swiglu(gate_up: torch.Tensor, suh: torch.Tensor,
                           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """xh[s] = fp16(H(silu(gate) * up * suh[s]) * 2^-4); gate_up bf16/fp16 [m, 2k] (gate first), suh fp16 [S, k]."""
    if gate_up.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("gate_up must be bf16 or fp16")
    _need(gate_up, gate_up.dtype, "gate_up")
    _need(suh, torch.float16, "suh")
    m, k2 = gate_up.shape
    if k2 % 2:
        raise ValueError("gate_up holds gate and up halves")
    k = k2 // 2
    s = suh.shape[0]
    if out is None:
        out = torch.empty((s, m, k), dtype=torch.float16, device=gate_up.device)
    _need(out, torch.float16, "out")
    st = lib().exl3_input_transform_swiglu(_ptr(gate_up), _BF16 if gate_up.dtype == torch.bfloat16 else _F16, m, k,
                                           _ptr(suh), s, _ptr(out), _stream(gate_up))
    _check(st, "exl3_input_transform_swiglu")
    return out


def moe_input_transform(x: torch.Tensor, sorted_ids: torch.Tensor, topk: int, block_expert: torch.Tensor,
                        block: int, suh: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gather and rotate block-aligned routed rows; suh fp16 [E, S, k] -> xh fp16 [S, rows, k]."""
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("x must be bf16 or fp16")
    _need(x, x.dtype, "x")
    _need(sorted_ids, torch.int32, "sorted_ids")
    _need(block_expert, torch.int32, "block_expert")
    _need(suh, torch.float16, "suh")
    num_tokens, k = x.shape
    e, s, _ = suh.shape
    rows = sorted_ids.numel()
    if out is None:
        out = torch.empty((s, rows, k), dtype=torch.float16, device=x.device)
    _need(out, torch.float16, "out")
    st = lib().exl3_moe_input_transform(_ptr(x), _BF16 if x.dtype == torch.bfloat16 else _F16, num_tokens, k,
                                        _ptr(sorted_ids), rows, int(topk), _ptr(block_expert), int(block), _ptr(suh),
                                        s, e, _ptr(out), _stream(x))
    _check(st, "exl3_moe_input_transform")
    return out


def moe_gemm(xh: torch.Tensor, trellis: torch.Tensor, bits: int, cb, svh: torch.Tensor, shard_cols: Sequence[int],
             block_expert: torch.Tensor, block: int, out_dtype=torch.bfloat16,
             out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Grouped GEMM; trellis int16 [E, k/16, n/16, 16*bits], svh fp16 [E, n] -> y [rows, n] (padded-row order)."""
    _need(xh, torch.float16, "xh")
    _need(trellis, torch.int16, "trellis")
    _need(svh, torch.float16, "svh")
    _need(block_expert, torch.int32, "block_expert")
    s, rows, k = xh.shape
    e, n = svh.shape
    if out is None:
        out = torch.empty((rows, n), dtype=out_dtype, device=xh.device)
    if out.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("output must be bf16 or fp16")
    _need(out, out.dtype, "out")
    cols, ns = _cols(shard_cols)
    cbid = CODEBOOKS[cb] if isinstance(cb, str) else int(cb)
    st = lib().exl3_moe_gemm(_ptr(xh), rows, k, _ptr(trellis), bits, cbid, _ptr(svh), cols, ns, _ptr(block_expert),
                             int(block), e, _ptr(out), _BF16 if out.dtype == torch.bfloat16 else _F16, n, _stream(xh))
    _check(st, "exl3_moe_gemm")
    return out


def moe_combine(y: torch.Tensor, sorted_ids: torch.Tensor, block_expert: torch.Tensor, block: int,
                num_experts: int, weights: torch.Tensor, topk: int, out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None, pair_rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Weighted sum of each token's top-k rows of a grouped GEMM's output:
    y [rows, n] (bf16/fp16), weights fp32 [tokens, topk] -> out [tokens, n].
    pair_rows is int32 [tokens * topk] scratch (allocated when not given)."""
    if y.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("y must be bf16 or fp16")
    _need(y, y.dtype, "y")
    _need(sorted_ids, torch.int32, "sorted_ids")
    _need(block_expert, torch.int32, "block_expert")
    _need(weights, torch.float32, "weights")
    rows, n = y.shape
    num_tokens = weights.shape[0]
    if weights.shape != (num_tokens, topk):
        raise ValueError("weights must be [tokens, topk]")
    if out is None:
        out = torch.empty((num_tokens, n), dtype=out_dtype, device=y.device)
    if out.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("output must be bf16 or fp16")
    _need(out, out.dtype, "out")
    if pair_rows is None:
        pair_rows = torch.empty(max(1, num_tokens * topk), dtype=torch.int32, device=y.device)
    _need(pair_rows, torch.int32, "pair_rows")
    st = lib().exl3_moe_combine(_ptr(y), _BF16 if y.dtype == torch.bfloat16 else _F16, rows, n, _ptr(sorted_ids),
                                _ptr(block_expert), int(block), int(num_experts), _ptr(weights), num_tokens,
                                int(topk), _ptr(pair_rows), _ptr(out), _BF16 if out.dtype == torch.bfloat16 else _F16,
                                _stream(y))
    _check(st, "exl3_moe_combine")
    return out


def _gemm_common(xh, trellis, bits, cb, svh, shard_cols, out_dtype, out):
    _need(xh, torch.float16, "xh")
    _need(trellis, torch.int16, "trellis")
    _need(svh, torch.float16, "svh")
    s, m, k = xh.shape
    n = int(shard_cols[-1])
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=xh.device)
    if out.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("output must be bf16 or fp16")
    _need(out, out.dtype, "out")
    cols, ns = _cols(shard_cols)
    if ns != s:
        raise ValueError("xh holds one slice per shard")
    cbid = CODEBOOKS[cb] if isinstance(cb, str) else int(cb)
    return m, k, n, cols, ns, cbid, out


def gemm(xh: torch.Tensor, trellis: torch.Tensor, bits: int, cb, svh: torch.Tensor, shard_cols: Sequence[int],
         out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    m, k, n, cols, ns, cbid, out = _gemm_common(xh, trellis, bits, cb, svh, shard_cols, out_dtype, out)
    st = lib().exl3_gemm(_ptr(xh), m, k, _ptr(trellis), bits, cbid, _ptr(svh), cols, ns, _ptr(out),
                         _BF16 if out.dtype == torch.bfloat16 else _F16, n, _stream(xh))
    _check(st, "exl3_gemm")
    return out


def gemm_splitk(xh: torch.Tensor, trellis: torch.Tensor, bits: int, cb, svh: torch.Tensor,
                shard_cols: Sequence[int], acc: torch.Tensor, out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Split-k variant; ``acc`` is an fp32 workspace of at least splitk_workspace_bytes (any contents;
    the call leaves it zeroed)."""
    m, k, n, cols, ns, cbid, out = _gemm_common(xh, trellis, bits, cb, svh, shard_cols, out_dtype, out)
    _need(acc, torch.float32, "acc")
    st = lib().exl3_gemm_splitk(_ptr(xh), m, k, _ptr(trellis), bits, cbid, _ptr(svh), cols, ns, _ptr(out),
                                _BF16 if out.dtype == torch.bfloat16 else _F16, n, _ptr(acc),
                                acc.numel() * 4, _stream(xh))
    _check(st, "exl3_gemm_splitk")
    return out


# Size of the library's built-in split-k scratch (EXL3_NOALLOC_SCRATCH_BYTES in include/exl3.h).
NOALLOC_SCRATCH_BYTES = 8 << 20


def gemm_splitk_noalloc(xh: torch.Tensor, trellis: torch.Tensor, bits: int, cb, svh: torch.Tensor,
                        shard_cols: Sequence[int], out_dtype=torch.bfloat16,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Split-k GEMM whose partials live in the library's built-in scratch array.

    For callers that cannot allocate a workspace.  Requests whose workspace
    would exceed NOALLOC_SCRATCH_BYTES are refused; calls must not overlap on
    the GPU (they share the one array).
    """
    m, k, n, cols, ns, cbid, out = _gemm_common(xh, trellis, bits, cb, svh, shard_cols, out_dtype, out)
    st = lib().exl3_gemm_splitk_noalloc(_ptr(xh), m, k, _ptr(trellis), bits, cbid, _ptr(svh), cols, ns, _ptr(out),
                                        _BF16 if out.dtype == torch.bfloat16 else _F16, n, _stream(xh))
    if st == 3:
        raise Exl3Error(st, f"exl3_gemm_splitk_noalloc (needs {splitk_workspace_bytes(m, k, n)} bytes of scratch, "
                            f"the built-in array holds {NOALLOC_SCRATCH_BYTES})")
    _check(st, "exl3_gemm_splitk_noalloc")
    return out


def linear(x: torch.Tensor, trellis: torch.Tensor, bits: int, cb, suh: torch.Tensor, svh: torch.Tensor,
           shard_cols: Sequence[int], out_dtype=torch.bfloat16, acc: Optional[torch.Tensor] = None,
           xh: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Whole layer: input rotation, then the GEMM (split-k when ``acc`` is given)."""
    xh = input_transform(x, suh, xh)
    if acc is not None:
        return gemm_splitk(xh, trellis, bits, cb, svh, shard_cols, acc, out_dtype, out)
    return gemm(xh, trellis, bits, cb, svh, shard_cols, out_dtype, out)


# Tile shapes exl3_test_gemm_shape accepts (EXL3_TEST_TILE_SHAPES in include/exl3.h).
TEST_TILE_SHAPES = 29


def test_gemm_shape(tile_shape: int, xh: torch.Tensor, trellis: torch.Tensor, bits: int, cb, svh: torch.Tensor,
                    shard_cols: Sequence[int], acc: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                    out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """exl3_gemm (or the split-k GEMM when ``acc`` is given) with a fixed tile shape.

    Returns None, launching nothing, when the shape cannot run the call.
    """
    m, k, n, cols, ns, cbid, out = _gemm_common(xh, trellis, bits, cb, svh, shard_cols, out_dtype, out)
    if acc is not None:
        _need(acc, torch.float32, "acc")
    st = lib().exl3_test_gemm_shape(int(tile_shape), _ptr(xh), m, k, _ptr(trellis), bits, cbid, _ptr(svh), cols, ns,
                                    _ptr(out), _BF16 if out.dtype == torch.bfloat16 else _F16, n,
                                    _ptr(acc) if acc is not None else None, acc.numel() * 4 if acc is not None else 0,
                                    _stream(xh))
    if st == 2:
        return None
    _check(st, "exl3_test_gemm_shape")
    return out


def test_codebook(cb, device="cuda") -> torch.Tensor:
    """fp16 bit patterns (as int16) of the codebook at all 65,536 states."""
    out = torch.empty(65536, dtype=torch.int16, device=device)
    cbid = CODEBOOKS[cb] if isinstance(cb, str) else int(cb)
    _check(lib().exl3_test_codebook(cbid, _ptr(out), _stream(out)), "exl3_test_codebook")
    return out


def test_unpack(trellis: torch.Tensor, bits: int, cb) -> torch.Tensor:
    """Dense Wq [k, n] (fp16 bit patterns as int16) decoded by the library."""
    _need(trellis, torch.int16, "trellis")
    kt, nt, w = trellis.shape
    if w != 16 * bits:
        raise ValueError("trellis last axis must be 16*bits")
    out = torch.empty((16 * kt, 16 * nt), dtype=torch.int16, device=trellis.device)
    cbid = CODEBOOKS[cb] if isinstance(cb, str) else int(cb)
    st = lib().exl3_test_unpack(_ptr(trellis), bits, cbid, 16 * kt, 16 * nt, _ptr(out), _stream(trellis))
    _check(st, "exl3_test_unpack")
    return out


# --------------------------------------------------------------------------------------------------
# rotary positions, the paged cache and attention

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}
KV_FORMATS = {"f16": 0, "bf16": 1, "int8": 2, "int4": 3}
_KV_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.uint8, "int4": torch.uint8}


# The current stream's handle, without a Stream object where torch has a call for that (not a public one).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _type(t: torch.Tensor, name: str) -> int:
    if t.dtype is torch.bfloat16:
        return _BF16
    if t.dtype is torch.float16:
        return _F16
    raise ValueError(f"{name} must be bf16 or fp16, got {t.dtype}")


def _heads(t: torch.Tensor, dtype, name: str) -> _Heads:
    """exl3_heads_t of a [tokens, heads, head_dim] view whose last axis is contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    ts, hs, ds = t.stride()
    tokens, heads, d = t.shape
    if ds != 1 and d > 1:
        raise ValueError(f"{name} must be contiguous along head_dim")
    # the stride of an axis of one (or no) element says nothing
    return _Heads(t.data_ptr(), ts if tokens > 1 else heads * d or 8, hs if heads > 1 else d)


def _one_device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    device = first.device
    for t in others:
        if t is not None and t.device != device:
            raise ValueError(f"tensors of one call must lie on one device: {device} and {t.device}")


def _comb(t: torch.Tensor):
    """(first byte, pieces, bytes from one to the next, bytes of one) that cover a view: its tokens, or with heads
    outermost its heads."""
    at, es = t.data_ptr(), t.element_size()
    if t.dim() == 3 and not t.is_contiguous():
        (n, h, d), (ts, hs, ds) = t.shape, t.stride()
        for pieces, step, others, stride in ((n, ts, h, hs), (h, hs, n, ts)):
            width = (others - 1) * stride + (d - 1) * ds + 1
            if width <= step:
                return at, pieces, step * es, width * es
    span = (1 + sum((n - 1) * st for n, st in zip(t.shape, t.stride()))) * es
    return at, 1, span, span


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two views share memory.  Views of different strides in one buffer may be taken to."""
    if a.numel() == 0 or b.numel() == 0:
        return False
    (a0, na, sa, wa), (b0, nb, sb, wb) = _comb(a), _comb(b)
    if a0 + (na - 1) * sa + wa <= b0 or b0 + (nb - 1) * sb + wb <= a0:
        return False
    if na > 1 and nb > 1 and sa != sb:
        return True
    # pieces i of a and i + k of b meet if -wb < b0 + k s - a0 < wa: the smallest k that passes the first
    s = sa if na > 1 else sb
    k = max(-(na - 1), (a0 - b0 - wb) // s + 1)
    return k < nb and b0 + k * s - a0 < wa


def _apart(out: torch.Tensor, name: str, **others) -> None:
    """Refuses an output that the caller gave if it shares memory with one of the call's other tensors."""
    for other, t in others.items():
        if t is not None and _overlap(out, t):
            raise ValueError(f"{name} overlaps {other}")


def _out_like(x: torch.Tensor, out: Optional[torch.Tensor], name: str):
    """The output of rows like x's and its exl3_heads_t; one that the caller gave is x itself or lies apart from it."""
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _, heads, d = x.shape
        return out, _Heads(out.data_ptr(), heads * d or 8, d)
    if out.shape != x.shape:
        raise ValueError(f"{name} must have the input's shape")
    oh = _heads(out, x.dtype, name)
    if oh.data != x.data_ptr() and _overlap(x, out):
        raise ValueError(f"{name} overlaps the input without being it")
    return out, oh


def _alike(t: torch.Tensor, dtype, shape, name: str) -> None:
    _need(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def rope_phases(rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0, fast: float = 32.0,
                slow: float = 1.0, original_len: float = 4096.0, device="cuda"):
    """(phases, amplitude) for rope and kv_write: int64 [rot_dim / 2] on ``device``, turns per position in 2^-64.

    scaling: "plain", "linear" (positions / factor), "ntk" (larger base) or "yarn" (slow frequencies / factor,
    fast ones kept, a ramp between ``slow`` and ``fast`` turns over ``original_len`` positions, as in the paper; code
    that ramps over the pairs' index gives other frequencies there: make such phases yourself).
    """
    out = torch.empty(max(0, int(rot_dim)) // 2, dtype=torch.int64)
    amplitude = ctypes.c_float(0.0)
    st = lib().exl3_rope_phases(int(rot_dim), float(base), ROPE_SCALINGS[scaling], float(factor), float(fast),
                                float(slow), float(original_len), out.data_ptr(), ctypes.byref(amplitude))
    _check(st, "exl3_rope_phases")
    return out.to(device), float(amplitude.value)


def _rope_args(positions: torch.Tensor, phases: torch.Tensor, layout: str, amplitude: float, tokens: int,
               axes: Optional[torch.Tensor] = None) -> _Rope:
    _need(phases, torch.int64, "phases")
    if axes is None:
        _alike(positions, torch.int32, (tokens,), "positions")
    elif positions.dim() != 2 or not 1 <= positions.shape[0] <= 255:
        raise ValueError("positions must be [axes, tokens] where axes are given")
    else:
        _alike(positions, torch.int32, (positions.shape[0], tokens), "positions")
        _alike(axes, torch.uint8, (phases.numel(),), "axes")
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    return _Rope(phases.data_ptr(), positions.data_ptr(), 2 * phases.numel(), ROPE_LAYOUTS[layout], float(amplitude))


def _axes_args(positions: torch.Tensor, axes: Optional[torch.Tensor]) -> Optional[_Axes]:
    return None if axes is None else _Axes(axes.data_ptr(), positions.shape[0])


def _norm_args(weight: Optional[torch.Tensor], eps: float, dtype, heads: int, d: int, name: str) -> Optional[_Norm]:
    """exl3_head_norm_t of weights [head_dim], the same for all heads, or [heads, head_dim]."""
    if weight is None:
        return None
    one = weight.dim() == 1
    _alike(weight, dtype, (d,) if one else (heads, d), name)
    return _Norm(weight.data_ptr(), 0 if one else d, float(eps))


def rope(x: torch.Tensor, positions: Optional[torch.Tensor] = None, phases: Optional[torch.Tensor] = None,
         layout: str = "half", amplitude: float = 1.0, out: Optional[torch.Tensor] = None,
         axes: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None, eps: float = 1e-6) -> torch.Tensor:
    """Rotary positions on the heads of x [tokens, heads, head_dim] (a view of a fused projection will do).

    The first 2 * phases.numel() values of every head turn.  ``out`` may be x itself.

    axes (uint8 [phases.numel()]): positions are int32 [number of axes, tokens], and pair i turns by the row axes[i] of
    them (time, height and width of images and video).  weight ([head_dim], or [heads, head_dim], of x's type): every
    head is first divided by sqrt(mean of its squares + eps) and multiplied by the weight, in the same pass and without
    a rounding in between; with a weight there need be no positions and phases, and nothing turns.
    """
    dt = _type(x, "x")
    xh = _heads(x, x.dtype, "x")
    tokens, heads, d = x.shape
    r = None
    if positions is not None and phases is not None:
        r = _rope_args(positions, phases, layout, amplitude, tokens, axes)
    elif weight is None or positions is not None or phases is not None or axes is not None:
        raise ValueError("x is only taken to be rotated or normed: it needs positions and phases, or a weight alone")
    norm = _norm_args(weight, eps, x.dtype, heads, d, "weight")
    _one_device(x, positions, phases, out, axes, weight)
    if out is not None and weight is not None:
        _apart(out, "out", weight=weight)
    out, oh = _out_like(x, out, "out")
    stream = _raw_stream(x.device.index)
    if norm is None and axes is None:
        st = lib().exl3_rope(xh, dt, tokens, heads, d, r, oh.data, oh.token_stride, oh.head_stride, stream)
        _check(st, "exl3_rope")
    else:
        st = lib().exl3_norm_rope(xh, dt, tokens, heads, d, norm, r, _axes_args(positions, axes), oh.data,
                                  oh.token_stride, oh.head_stride, stream)
        _check(st, "exl3_norm_rope")
    return out


class KVCache:
    """A paged cache: k and v [pages, kv_heads, page_size, row] (row: head_dim values in 16 bits, head_dim bytes for
    "int8", head_dim / 2 for "int4"), and for the quantised formats bf16 scales [pages, kv_heads, page_size].

    The calls take the addresses of these tensors as they were at construction, so the attributes cannot be assigned:
    other tensors are another KVCache (which costs a few checks and no copy)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor],
                 v_scale: Optional[torch.Tensor], fmt: str):
        if fmt not in KV_FORMATS:
            raise ValueError(f"cache format must be one of {sorted(KV_FORMATS)}")
        dtype = _KV_DTYPES[fmt]
        _need(k, dtype, "k")
        if k.dim() != 4:
            raise ValueError("k must be [pages, kv_heads, page_size, row]")
        _alike(v, dtype, k.shape, "v")
        pages, heads, page, row = k.shape
        if fmt in ("int8", "int4"):
            if k_scale is None or v_scale is None:
                raise ValueError(f"an {fmt} cache needs scales")
            _alike(k_scale, torch.bfloat16, (pages, heads, page), "k_scale")
            _alike(v_scale, torch.bfloat16, (pages, heads, page), "v_scale")
        _one_device(k, v, k_scale, v_scale)
        head_dim = 2 * row if fmt == "int4" else row
        args = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if k_scale is not None else None,
                      v_scale.data_ptr() if v_scale is not None else None, pages, page, heads, head_dim,
                      KV_FORMATS[fmt])
        self.__dict__.update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, fmt=fmt, num_pages=pages, kv_heads=heads,
                             page_size=page, head_dim=head_dim, args=args)

    def __setattr__(self, name, value):
        raise AttributeError(f"KVCache.{name} cannot be assigned: make a KVCache of the new tensors")

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, fmt: str, device="cuda") -> "KVCache":
        """A cache of rows not yet written."""
        if fmt not in KV_FORMATS:
            raise ValueError(f"cache format must be one of {sorted(KV_FORMATS)}")
        shape = (num_pages, kv_heads, page_size, head_dim // 2 if fmt == "int4" else head_dim)
        k, v = (torch.zeros(shape, dtype=_KV_DTYPES[fmt], device=device) for _ in range(2))
        scales = [None, None]
        if fmt in ("int8", "int4"):
            scales = [torch.ones(shape[:3], dtype=torch.bfloat16, device=device) for _ in range(2)]
        return cls(k, v, scales[0], scales[1], fmt)


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, q: Optional[torch.Tensor] = None,
             positions: Optional[torch.Tensor] = None, phases: Optional[torch.Tensor] = None, layout: str = "half",
             amplitude: float = 1.0, q_out: Optional[torch.Tensor] = None, axes: Optional[torch.Tensor] = None,
             q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
             eps: float = 1e-6) -> Optional[torch.Tensor]:
    """Write k and v [tokens, kv_heads, head_dim] into the cache rows ``slots`` (int64; page * page_size + row,
    anything outside the cache writes nothing).

    With positions and phases the keys are rotated first, and so is q [tokens, heads, head_dim] when given: the
    rotated q (q_out, a new tensor unless given) is returned, else None.

    axes: positions are [number of axes, tokens], as for rope.  q_weight, k_weight ([head_dim], or [heads, head_dim]):
    the heads of q and k are first divided by their root mean square and multiplied by these, as for rope; with
    q_weight q needs no positions.
    """
    dt = _type(k, "k")
    tokens = k.shape[0]
    kh, vh = _heads(k, k.dtype, "k"), _heads(v, k.dtype, "v")
    if tuple(k.shape) != (tokens, cache.kv_heads, cache.head_dim) or v.shape != k.shape:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] of the cache")
    _alike(slots, torch.int64, (tokens,), "slots")
    _one_device(k, v, cache.k, slots, q, positions, phases, q_out, axes, q_weight, k_weight)
    r = qh = None
    heads, qo = 0, (None, 0, 0)
    if phases is not None:
        if positions is None:
            raise ValueError("phases need positions")
        r = _rope_args(positions, phases, layout, amplitude, tokens, axes)
    elif axes is not None:
        raise ValueError("axes need positions and phases")
    kn = _norm_args(k_weight, eps, k.dtype, cache.kv_heads, cache.head_dim, "k_weight")
    qn = None
    if q is not None:
        if r is None and q_weight is None:
            raise ValueError("q is only taken to be rotated or normed: it needs positions and phases, or q_weight")
        if q.dim() != 3 or q.shape[0] != tokens or q.shape[2] != cache.head_dim:
            raise ValueError("q must be [tokens, heads, head_dim]")
        qh, heads = _heads(q, k.dtype, "q"), q.shape[1]
        qn = _norm_args(q_weight, eps, k.dtype, heads, cache.head_dim, "q_weight")
        if q_out is not None:
            _apart(q_out, "q_out", k=k, v=v, cache_k=cache.k, cache_v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale,
                   q_weight=q_weight, k_weight=k_weight)
        q_out, oh = _out_like(q, q_out, "q_out")
        qo = (oh.data, oh.token_stride, oh.head_stride)
    elif q_out is not None or q_weight is not None:
        raise ValueError(("q_out" if q_out is not None else "q_weight") + " without q")
    stream = _raw_stream(k.device.index)
    if qn is None and kn is None and axes is None:
        st = lib().exl3_kv_write(cache.args, kh, vh, dt, tokens, slots.data_ptr(), r, qh, heads, *qo, stream)
        _check(st, "exl3_kv_write")
    else:
        st = lib().exl3_norm_kv_write(cache.args, kh, vh, dt, tokens, slots.data_ptr(), qn, kn, r,
                                      _axes_args(positions, axes), qh, heads, *qo, stream)
        _check(st, "exl3_norm_kv_write")
    return q_out


def kv_read(cache: KVCache, slots: torch.Tensor, dtype=torch.bfloat16, k: Optional[torch.Tensor] = None,
            v: Optional[torch.Tensor] = None):
    """(k, v) [tokens, kv_heads, head_dim] of the cache rows ``slots``; zeros for a slot outside the cache."""
    _need(slots, torch.int64, "slots")
    if slots.dim() != 1:
        raise ValueError("slots must be [tokens]")
    _one_device(slots, cache.k, k, v)
    shape = (slots.numel(), cache.kv_heads, cache.head_dim)
    if k is not None:
        _apart(k, "k", cache_k=cache.k, cache_v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale, v=v)
    if v is not None:
        _apart(v, "v", cache_k=cache.k, cache_v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale)
    k = torch.empty(shape, dtype=dtype, device=slots.device) if k is None else k
    v = torch.empty(shape, dtype=dtype, device=slots.device) if v is None else v
    _alike(k, dtype, shape, "k")
    _alike(v, dtype, shape, "v")
    st = lib().exl3_kv_read(cache.args, slots.data_ptr(), shape[0], _type(k, "k"), k.data_ptr(), v.data_ptr(), _raw_stream(slots.device.index))
    _check(st, "exl3_kv_read")
    return k, v


class KVTables:
    """Page tables of a batch of requests on the GPU, and the free pages of a cache as a stack.

    block_table int32 [batch, width], kv_lens int32 [batch] (cached tokens), held int32 [batch] (pages in the table's row),
    free_pages int32 [capacity], of which the first free_count (int32 [1]) are free.  kv_lens may be set back (refused
    drafts) without touching held.  As with KVCache, the calls take the addresses that the tensors have now."""

    def __init__(self, block_table: torch.Tensor, kv_lens: torch.Tensor, held: torch.Tensor, free_pages: torch.Tensor,
                 free_count: torch.Tensor, page_size: int):
        _need(block_table, torch.int32, "block_table")
        if block_table.dim() != 2 or block_table.shape[1] < 1:
            raise ValueError("block_table must be [batch, width]")
        batch, width = block_table.shape
        _alike(kv_lens, torch.int32, (batch,), "kv_lens")
        _alike(held, torch.int32, (batch,), "held")
        _need(free_pages, torch.int32, "free_pages")
        if free_pages.dim() != 1 or not 1 <= free_pages.numel() < 1 << 30:
            raise ValueError("free_pages must be [capacity], below 2^30")
        _alike(free_count, torch.int32, (1,), "free_count")
        _one_device(block_table, kv_lens, held, free_pages, free_count)
        if page_size not in (16, 32, 64, 128, 256) or width * page_size > 1 << 30:
            raise ValueError("page_size must be 16, 32, 64, 128 or 256, and a row of the table at most 2^30 tokens")
        parts = {"block_table": block_table, "kv_lens": kv_lens, "held": held, "free_pages": free_pages, "free_count": free_count}
        names = list(parts)
        for i, name in enumerate(names):
            _apart(parts[name], name, **{n: parts[n] for n in names[i + 1:]})
        args = _Tables(block_table.data_ptr(), kv_lens.data_ptr(), held.data_ptr(), free_pages.data_ptr(),
                       free_count.data_ptr(), batch, width, page_size, free_pages.numel())
        spans = tuple((t.data_ptr(), t.data_ptr() + 4 * t.numel()) for t in (kv_lens, held, free_count))
        same = (block_table.data_ptr(), free_pages.data_ptr(), batch, width, page_size, free_pages.numel())
        self.__dict__.update(parts, batch=batch, table_width=width, page_size=page_size, args=args, _spans=spans, _same=same,
                             _outs=tuple(at for at, _ in spans))

    def __setattr__(self, name, value):
        raise AttributeError(f"KVTables.{name} cannot be assigned: make a KVTables of the new tensors")

    @classmethod
    def empty(cls, batch: int, max_len: int, num_pages: int, page_size: int, device="cuda") -> "KVTables":
        """Tables of requests without tokens, each with room for max_len, over a cache of num_pages free pages."""
        width = max(1, (max_len + page_size - 1) // page_size)

        def ints(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)

        free = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)  # page 0 is taken first
        return cls(ints(batch, width) - 1, ints(batch), ints(batch), free, ints(1) + num_pages, page_size)


def _new_state(tables: KVTables, into: Optional[KVTables]) -> KVTables:
    """Where a call writes the new lengths, held pages and count: the tables' own, or those of another KVTables over the
    same table and stack."""
    if into is None or into is tables:
        return tables
    if into._same != tables._same:
        raise ValueError("into must share block_table and free_pages with the tables")
    for i, (a0, a1) in enumerate(into._spans):
        for j, (b0, b1) in enumerate(tables._spans):
            if a0 < b1 and b0 < a1 and (i != j or a0 != b0):
                raise ValueError("into overlaps the tables without being in their place")
    return into


def kv_plan(tables: KVTables, new_lens: torch.Tensor, total: int, into: Optional[KVTables] = None,
            cu_q: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
            slots: Optional[torch.Tensor] = None, granted: Optional[torch.Tensor] = None):
    """(cu_q, positions, slots, granted): a step's packing of new_lens[b] (int32 [batch]) new tokens of each request, and
    pages for them, all on the GPU.

    cu_q int32 [batch + 1]; positions int32 [total] and slots int64 [total] of the packed tokens (rows past the last
    token: position 0 and slot -1, so ``total`` may be the fixed size of a captured step); granted bool [batch].  The
    tables' lengths, rows and stack move on, or with ``into`` (a KVTables over the same block_table and free_pages) the
    new lengths, held pages and count go there.  A request whose pages are not to be had (or whose tokens do not fit
    into total, or pages into the table) is not granted: its state stays and its slots are -1; none after it gets
    pages that it waits for.  Attention's outputs for its rows mean nothing.  The four outputs are new tensors unless given.
    """
    total, batch = int(total), tables.batch
    device = tables.kv_lens.device
    _alike(new_lens, torch.int32, (batch,), "new_lens")
    state = tables if into is None else _new_state(tables, into)
    if not (cu_q is None and positions is None and slots is None and granted is None):
        given = {"cu_q": cu_q, "positions": positions, "slots": slots, "granted": granted}
        shapes = {"cu_q": (torch.int32, batch + 1), "positions": (torch.int32, total), "slots": (torch.int64, total),
                  "granted": (torch.bool, batch)}
        seen = dict(_state_parts(tables, state), new_lens=new_lens)
        for name, t in given.items():
            if t is not None:
                _alike(t, shapes[name][0], (shapes[name][1],), name)
                _apart(t, name, **seen)
                seen[name] = t
    rows = max(0, total)
    cu_q = torch.empty(batch + 1, dtype=torch.int32, device=device) if cu_q is None else cu_q
    positions = torch.empty(rows, dtype=torch.int32, device=device) if positions is None else positions
    slots = torch.empty(rows, dtype=torch.int64, device=device) if slots is None else slots
    granted = torch.empty(batch, dtype=torch.bool, device=device) if granted is None else granted
    _one_device(tables.kv_lens, new_lens, state.kv_lens, cu_q, positions, slots, granted)
    st = lib().exl3_kv_plan(tables.args, new_lens.data_ptr(), total, *state._outs, cu_q.data_ptr(), positions.data_ptr(),
                            slots.data_ptr(), granted.data_ptr(), _raw_stream(device.index))
    _check(st, "exl3_kv_plan")
    return cu_q, positions, slots, granted


def _state_parts(tables: KVTables, state: KVTables) -> dict:
    parts = {n: getattr(tables, n) for n in ("block_table", "kv_lens", "held", "free_pages", "free_count")}
    if state is not tables:
        parts.update({"into_" + n: getattr(state, n) for n in ("kv_lens", "held", "free_count")})
    return parts


def kv_release(tables: KVTables, ended: torch.Tensor, shared: Optional[torch.Tensor] = None,
               into: Optional[KVTables] = None) -> None:
    """Requests end (bool [batch]): their pages go back onto the stack, their lengths and held pages become 0.

    shared (int32 [batch]): leading pages of an ended request's row that belong to others too and stay off the stack.
    ``into`` as for kv_plan.
    """
    _alike(ended, torch.bool, (tables.batch,), "ended")
    if shared is not None:
        _alike(shared, torch.int32, (tables.batch,), "shared")
    state = _new_state(tables, into)
    _one_device(tables.kv_lens, ended, shared, state.kv_lens)
    st = lib().exl3_kv_release(tables.args, ended.data_ptr(), None if shared is None else shared.data_ptr(), *state._outs,
                               _raw_stream(tables.kv_lens.device.index))
    _check(st, "exl3_kv_release")


def attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, max_len: int = 0,
                     scale: Optional[float] = None, window: int = 0,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention over packed prompts: q [total, heads, head_dim], k and v [total, kv_heads, head_dim],
    sequence b the tokens cu_seqlens[b] .. cu_seqlens[b + 1] (int32).

    scale: 1 / sqrt(head_dim) unless given.  window > 0: a query sees its own and the window - 1 keys before.
    max_len is accepted for symmetry with attention_paged; the split does not need it.
    """
    dt = _type(q, "q")
    qh, kh, vh = _heads(q, q.dtype, "q"), _heads(k, q.dtype, "k"), _heads(v, q.dtype, "v")
    total, heads, d = q.shape
    if k.shape[0] != total or k.shape[2] != d or v.shape != k.shape:
        raise ValueError("k and v must be [total, kv_heads, head_dim]")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [batch + 1]")
    _one_device(q, k, v, cu_seqlens, out)
    if out is not None:
        _apart(out, "out", k=k, v=v)
    out, oh = _out_like(q, out, "out")
    st = lib().exl3_attention_prompt(qh, kh, vh, dt, total, heads, k.shape[1], d, cu_seqlens.data_ptr(),
                                     cu_seqlens.numel() - 1, int(window), d ** -0.5 if scale is None else float(scale),
                                     oh.data, oh.token_stride, oh.head_stride, _raw_stream(q.device.index))
    _check(st, "exl3_attention_prompt")
    return out


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(*sizes) -> int:
    return int(lib().exl3_attention_paged_workspace_bytes(*sizes))


def attention_paged_workspace_bytes(total_q: int, batch: int, heads: int, kv_heads: int, head_dim: int, max_q: int,
                                    max_kv: int, window: int = 0) -> int:
    return _workspace_bytes(total_q, batch, heads, kv_heads, head_dim, max_q, max_kv, window)


def attention_paged(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, cu_q: torch.Tensor,
                    kv_lens: torch.Tensor, max_q: int, max_kv: int, scale: Optional[float] = None, window: int = 0,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of each sequence's last tokens over the cache, their own rows already written.

    q [total_q, heads, head_dim], packed by cu_q (int32 [batch + 1]); block_table int32 [batch, width]; kv_lens int32
    [batch]; max_q and max_kv: the largest of the sequences' query and cached tokens (max_q must not be too small).
    ``workspace``: uint8, at least attention_paged_workspace_bytes (allocated when not given).
    """
    dt = _type(q, "q")
    qh = _heads(q, q.dtype, "q")
    total, heads, d = q.shape
    if d != cache.head_dim:
        raise ValueError("q and the cache differ in head_dim")
    _need(cu_q, torch.int32, "cu_q")
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be [batch + 1]")
    batch = cu_q.numel() - 1
    _alike(kv_lens, torch.int32, (batch,), "kv_lens")
    _need(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError("block_table must be [batch, width]")
    _one_device(q, cache.k, block_table, cu_q, kv_lens, out, workspace)
    if out is not None:
        _apart(out, "out", cache_k=cache.k, cache_v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale)
    out, oh = _out_like(q, out, "out")
    if workspace is None:
        need = _workspace_bytes(total, batch, heads, cache.kv_heads, d, int(max_q), int(max_kv), int(window))
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _need(workspace, torch.uint8, "workspace")
    st = lib().exl3_attention_paged(qh, dt, total, heads, cache.args, block_table.data_ptr(), block_table.shape[1],
                                cu_q.data_ptr(), kv_lens.data_ptr(), batch, int(max_q), int(max_kv), int(window),
                                d ** -0.5 if scale is None else float(scale), oh.data, oh.token_stride,
                                oh.head_stride, workspace.data_ptr(), workspace.numel(), _raw_stream(q.device.index))
    _check(st, "exl3_attention_paged")
    return out


SHARE_ALWAYS = 2**31 - 1  # EXL3_SHARE_ALWAYS in include/exl3.h


@functools.lru_cache(maxsize=1024)
def _shared_workspace_bytes(*sizes) -> int:
    return int(lib().exl3_attention_shared_workspace_bytes(*sizes))


@functools.lru_cache(maxsize=1024)
def _sharing_pays(*sizes) -> bool:
    return bool(lib().exl3_attention_shared_pays(*sizes))


def _steer(total_q: int, batch: int, sharers: Optional[int], groups: int, heads: int, dtype, cache: KVCache, max_q: int,
           max_prefix: int) -> int:
    """max_prefix, or 0 (not shared) where sharing does not pay for so many of the sequences."""
    if sharers is None:
        return max_prefix
    sharers = int(sharers)
    if not 0 <= sharers <= batch:
        raise ValueError("sharers must be a number of the call's sequences")
    if max_prefix == SHARE_ALWAYS or _sharing_pays(total_q, batch, sharers, groups, heads, cache.kv_heads, cache.head_dim,
                                                   _BF16 if dtype is torch.bfloat16 else _F16, KV_FORMATS[cache.fmt],
                                                   max_q, max_prefix):
        return max_prefix
    return 0


def attention_shared_workspace_bytes(total_q: int, batch: int, groups: int, heads: int, dtype, cache: KVCache, max_q: int,
                                     max_kv: int, max_prefix: int, sharers: Optional[int] = None) -> int:
    """dtype: q's."""
    max_prefix = _steer(total_q, batch, sharers, groups, heads, dtype, cache, max_q, max_prefix)
    return _shared_workspace_bytes(total_q, batch, groups, heads, cache.kv_heads, cache.head_dim,
                                   _BF16 if dtype is torch.bfloat16 else _F16, KV_FORMATS[cache.fmt], max_q, max_kv, max_prefix)


def attention_shared(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, cu_q: torch.Tensor,
                     kv_lens: torch.Tensor, cu_groups: torch.Tensor, prefix_lens: torch.Tensor, max_q: int, max_kv: int,
                     max_prefix: int, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, sharers: Optional[int] = None) -> torch.Tensor:
    """attention_paged for sequences that begin with the same cached tokens, which are read once for all of them.

    Group g is the sequences cu_groups[g] .. cu_groups[g + 1] - 1 (int32 [groups + 1]; sequences outside are of no
    group), whose first prefix_lens[g] (int32 [groups]) keys and values are the same and are read through the table of
    the first of them that has queries.  Shared are the keys that every query of the group sees (rows that kv_plan did
    not grant see fewer).  Over a quantised cache the rows, keys and values of the prefix are rounded as in long chunks.
    max_prefix: about the longest of the prefixes, which steers whether they are shared (for few sequences or short
    prefixes the call is attention_paged; SHARE_ALWAYS: they are; 0: they are not).  sharers: how many sequences the
    groups hold, all unless given; where they are fewer, sharing must pay for those.
    ``workspace``: uint8, at least attention_shared_workspace_bytes (allocated when not given).
    Other arguments as for attention_paged.
    """
    dt = _type(q, "q")
    qh = _heads(q, q.dtype, "q")
    total, heads, d = q.shape
    if d != cache.head_dim:
        raise ValueError("q and the cache differ in head_dim")
    _need(cu_q, torch.int32, "cu_q")
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be [batch + 1]")
    batch = cu_q.numel() - 1
    _alike(kv_lens, torch.int32, (batch,), "kv_lens")
    _need(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError("block_table must be [batch, width]")
    _need(cu_groups, torch.int32, "cu_groups")
    if cu_groups.dim() != 1 or cu_groups.numel() < 1:
        raise ValueError("cu_groups must be [groups + 1]")
    groups = cu_groups.numel() - 1
    _alike(prefix_lens, torch.int32, (groups,), "prefix_lens")
    _one_device(q, cache.k, block_table, cu_q, kv_lens, cu_groups, prefix_lens, out, workspace)
    if out is not None:
        _apart(out, "out", cache_k=cache.k, cache_v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale)
    out, oh = _out_like(q, out, "out")
    max_prefix = _steer(total, batch, sharers, groups, heads, q.dtype, cache, int(max_q), int(max_prefix))
    if workspace is None:
        need = attention_shared_workspace_bytes(total, batch, groups, heads, q.dtype, cache, int(max_q), int(max_kv), int(max_prefix))
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _need(workspace, torch.uint8, "workspace")
    st = lib().exl3_attention_shared(qh, dt, total, heads, cache.args, block_table.data_ptr(), block_table.shape[1],
                                     cu_q.data_ptr(), kv_lens.data_ptr(), batch, cu_groups.data_ptr(),
                                     prefix_lens.data_ptr(), groups, int(max_q), int(max_kv), int(max_prefix),
                                     d ** -0.5 if scale is None else float(scale), oh.data, oh.token_stride,
                                     oh.head_stride, workspace.data_ptr(), workspace.numel(), _raw_stream(q.device.index))
    _check(st, "exl3_attention_shared")
    return out
