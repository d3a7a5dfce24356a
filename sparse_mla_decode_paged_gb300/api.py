"""Thin PyTorch binding of the C ABI: argument marshalling only.

Every step of the decode runs in the CUDA library; torch provides device
memory and the current stream.  Names follow include/sparse_mla.h.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Tuple

import torch

from . import _native
from ._native import (SmlaAppendDims, SmlaDenseDims, SmlaDensePlan, SmlaDims, SmlaNormAppendDims, SmlaNormRopeDims,
                      SmlaPlan, SmlaTopkDims, check)

PAGE_SIZE, D_LATENT, D_ROPE, D_QK = 64, 512, 64, 576


def _lib():
    return _native.load()


def _ptr(t: Optional[torch.Tensor]):
    """Device address for a void* argument (the library's argument types convert a plain int)."""
    return t.data_ptr() if t is not None else None


def _stream(stream=None):
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _need(t: torch.Tensor, name: str, dtype, ndim: int):
    # the common case in one expression; the checks below only name what is wrong
    if type(t) is torch.Tensor and t.is_cuda and t.dtype is dtype and t.dim() == ndim and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


MERGE_AUTO, MERGE_KERNEL, MERGE_FUSED = 0, 1, 2


def make_dims(B: int, H: int, topk: int, max_pages_per_seq: int, num_pages: int, nsplit: int = 0,
              heads_per_cta: int = 0, queries_per_request: int = 1, merge: int = MERGE_AUTO) -> SmlaDims:
    return SmlaDims(B, H, topk, PAGE_SIZE, max_pages_per_seq, D_LATENT, D_ROPE, nsplit, num_pages, heads_per_cta,
                    queries_per_request, merge)


def dims_of(q, kv_cache, block_table, topk_idx, nsplit: int = 0, heads_per_cta: int = 0,
            merge: int = MERGE_AUTO) -> SmlaDims:
    """Shapes of a call; several queries per request when q has a multiple of block_table's rows."""
    return make_dims(q.shape[0], q.shape[1], topk_idx.shape[1], block_table.shape[1], kv_cache.shape[0], nsplit,
                     heads_per_cta, q.shape[0] // block_table.shape[0], merge)


# Decode dims by call shape and device, with the split count the library's scheduler chose filled in: a
# call with the same shapes as an earlier one reuses them (the library reads dims, never writes them).
_DECODE_DIMS = {}


def _decode_dims(q, kv_cache, block_table, topk_idx, nsplit: int, heads_per_cta: int, merge: int) -> SmlaDims:
    key = (q.shape, kv_cache.shape[0], block_table.shape, topk_idx.shape[1], nsplit, heads_per_cta, merge,
           q.device.index)
    d = _DECODE_DIMS.get(key)
    if d is None:
        d = dims_of(q, kv_cache, block_table, topk_idx, nsplit, heads_per_cta, merge)
        if nsplit == 0:
            d.nsplit = plan(d, q.device.index).nsplit
        if len(_DECODE_DIMS) > 256:
            _DECODE_DIMS.clear()
        _DECODE_DIMS[key] = d
    return d


def plan_for(dims: SmlaDims, sm_count: int) -> SmlaPlan:
    p = SmlaPlan()
    check("sparse_mla_plan_for", _lib().sparse_mla_plan_for(C.byref(dims), sm_count, C.byref(p)))
    return p


def plan(dims: SmlaDims, device: Optional[int] = None) -> SmlaPlan:
    p = SmlaPlan()
    dev = torch.cuda.current_device() if device is None else device
    check("sparse_mla_plan", _lib().sparse_mla_plan(C.byref(dims), dev, C.byref(p)))
    return p


def workspace_size(dims: SmlaDims, nsplit: int) -> int:
    return int(_lib().sparse_mla_workspace_size(C.byref(dims), nsplit))


def alloc_workspace(dims: SmlaDims, nsplit: int, device=None) -> torch.Tensor:
    """Caller-owned workspace (zeroed, so the device error word starts clear)."""
    n = workspace_size(dims, nsplit)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _check_inputs(q, kv_cache, block_table, topk_idx, seq_lens):
    _need(q, "q", torch.bfloat16, 3)
    _need(kv_cache, "kv_cache", torch.uint8, 3)
    _need(block_table, "block_table", torch.int32, 2)
    _need(topk_idx, "topk_idx", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    if q.shape[2] != D_QK or kv_cache.shape[1] != PAGE_SIZE or kv_cache.shape[2] != 656:
        raise ValueError("q must be [B,H,576] and kv_cache [pages,64,656]")
    B = q.shape[0]
    R = block_table.shape[0]
    if R < 1 or B % R != 0 or topk_idx.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("q, topk_idx and seq_lens need one row per query, block_table one row per request "
                         "(a divisor of the query count)")


def sparse_mla_decode(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor, topk_idx: torch.Tensor,
                      seq_lens: torch.Tensor, sm_scale: float, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      nsplit: int = 0, stream=None, heads_per_cta: int = 0,
                      merge: int = MERGE_AUTO) -> Tuple[torch.Tensor, torch.Tensor]:
    """out bf16 [B,H,512], lse fp32 [B,H].  nsplit = 0, heads_per_cta = 0 and merge = MERGE_AUTO let the
    library's scheduler choose."""
    _check_inputs(q, kv_cache, block_table, topk_idx, seq_lens)
    dims = _decode_dims(q, kv_cache, block_table, topk_idx, nsplit, heads_per_cta, merge)
    if out is None:
        out = torch.empty((q.shape[0], q.shape[1], D_LATENT), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((q.shape[0], q.shape[1]), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(dims, dims.nsplit, q.device)
    st = _lib().sparse_mla_decode(
        dims, q.data_ptr(), kv_cache.data_ptr(), block_table.data_ptr(), topk_idx.data_ptr(), seq_lens.data_ptr(),
        sm_scale, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(stream))
    if st != 0:
        check("sparse_mla_decode", st)
    return out, lse


def sparse_mla_decode_rows(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                           topk_idx: torch.Tensor, seq_lens: torch.Tensor, sm_scale: float,
                           workspace: Optional[torch.Tensor] = None, nsplit: int = 0, stream=None,
                           heads_per_cta: int = 0, rows: Optional[torch.Tensor] = None, merge: int = MERGE_AUTO):
    """sparse_mla_decode that also returns the rows the decode's split kernel loaded:
    (out bf16 [B,H,512], lse fp32 [B,H], rows int64 [B,topk], -1 for skipped entries)."""
    _check_inputs(q, kv_cache, block_table, topk_idx, seq_lens)
    B, H = q.shape[0], q.shape[1]
    dims = dims_of(q, kv_cache, block_table, topk_idx, nsplit, heads_per_cta, merge)
    if nsplit == 0:
        nsplit = plan(dims, q.device.index).nsplit
        dims.nsplit = nsplit
    out = torch.empty((B, H, D_LATENT), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if rows is None:
        rows = torch.empty(topk_idx.shape, dtype=torch.int64, device=q.device)
    _need(rows, "rows", torch.int64, 2)
    if workspace is None:
        workspace = alloc_workspace(dims, nsplit, q.device)
    check("sparse_mla_decode_rows", _lib().sparse_mla_decode_rows(
        C.byref(dims), _ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(topk_idx), _ptr(seq_lens),
        C.c_float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace), C.c_size_t(workspace.numel()),
        _ptr(rows), _stream(stream)))
    return out, lse, rows


def debug_set_wait_limit(ns: int) -> None:
    """Time limit of the split kernel's pipeline waits for later launches (0 = the default, 1 s)."""
    check("sparse_mla_debug_set_wait_limit", _lib().sparse_mla_debug_set_wait_limit(int(ns)))


def sparse_mla_split(q, kv_cache, block_table, topk_idx, seq_lens, sm_scale: float, nsplit: int,
                     err_word: Optional[torch.Tensor] = None, stream=None, heads_per_cta: int = 0):
    """Partials: o_part fp32 [B,nsplit,H,512], lse_part fp32 [B,nsplit,H]."""
    _check_inputs(q, kv_cache, block_table, topk_idx, seq_lens)
    B, H = q.shape[0], q.shape[1]
    dims = dims_of(q, kv_cache, block_table, topk_idx, nsplit, heads_per_cta)
    o_part = torch.empty((B, nsplit, H, D_LATENT), dtype=torch.float32, device=q.device)
    lse_part = torch.empty((B, nsplit, H), dtype=torch.float32, device=q.device)
    check("sparse_mla_split", _lib().sparse_mla_split(
        C.byref(dims), nsplit, _ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(topk_idx), _ptr(seq_lens),
        C.c_float(sm_scale), _ptr(o_part), _ptr(lse_part), _ptr(err_word), _stream(stream)))
    return o_part, lse_part


def sparse_mla_kv_append(latent: torch.Tensor, rope: torch.Tensor, block_table: torch.Tensor,
                         positions: torch.Tensor, kv_cache: torch.Tensor, requests: Optional[torch.Tensor] = None,
                         err_word: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise new tokens (latent bf16 [T,512], rope bf16 [T,64]) into the paged FP8 cache at
    (requests[i] or i, positions[i]) through block_table; kv_cache is written in place."""
    _need(latent, "latent", torch.bfloat16, 2)
    _need(rope, "rope", torch.bfloat16, 2)
    _need(block_table, "block_table", torch.int32, 2)
    _need(positions, "positions", torch.int32, 1)
    _need(kv_cache, "kv_cache", torch.uint8, 3)
    T = latent.shape[0]
    if latent.shape[1] != D_LATENT or rope.shape != (T, D_ROPE) or positions.shape[0] != T:
        raise ValueError("latent must be [T,512], rope [T,64], positions [T]")
    if kv_cache.shape[1] != PAGE_SIZE or kv_cache.shape[2] != 656:
        raise ValueError("kv_cache must be [pages,64,656]")
    if requests is not None:
        _need(requests, "requests", torch.int32, 1)
        if requests.shape[0] != T:
            raise ValueError("requests must be [T]")
    dims = SmlaAppendDims(T, block_table.shape[0], PAGE_SIZE, block_table.shape[1], D_LATENT, D_ROPE,
                          kv_cache.shape[0])
    check("sparse_mla_kv_append", _lib().sparse_mla_kv_append(
        C.byref(dims), _ptr(latent), _ptr(rope), _ptr(block_table), _ptr(requests), _ptr(positions),
        _ptr(kv_cache), _ptr(err_word), _stream(stream)))


# ----------------------------------------------------------------------------- around the paged cache

_DTYPE = {torch.bfloat16: _native.BF16, torch.float16: _native.FP16, torch.float32: _native.FP32}


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _err_word(t, dev):
    if t is not None:
        _need(t, "err_word", torch.int32, 1)
        if t.numel() < 1 or t.device != dev:
            raise ValueError(f"err_word must hold one int32 on {dev}")
    return _ptr(t)


class _on:
    """The stream a call launches on (the caller's, or its device's current one), with the tensors' device
    current and, for a stream of the caller's, allocations made on it."""
    __slots__ = ("raw", "ctx")

    def __init__(self, dev, stream=None):
        self.ctx = None
        if stream is None:
            self.raw = torch._C._cuda_getCurrentRawStream(dev.index)      # current_stream(dev) without its object
            if dev.index != torch.cuda.current_device():
                self.ctx = torch.cuda.device(dev)
        else:
            if stream.device != dev:
                raise ValueError(f"stream must belong to {dev}, got {stream.device}")
            self.raw = stream.cuda_stream
            self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.raw

    def __exit__(self, *a):
        if self.ctx is not None:
            self.ctx.__exit__(*a)


# Dims of calls whose arguments have been checked, by the shapes, strides, types and devices of the tensors and the
# values that the checks look at (the library reads dims, never writes them).
_CHECKED = {}


def _call_key(tensors, *values):
    """None when one of the tensors is something else: the checks name it."""
    try:
        return (tuple([t if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in tensors]), values)
    except (AttributeError, TypeError):
        return None


def _remember(key, checked):
    if key is not None:
        if len(_CHECKED) > 256:
            _CHECKED.clear()
        _CHECKED[key] = checked
    return checked


def rope_table(max_positions: int, rope_dim: int = D_ROPE, base: float = 10000.0, device=None) -> torch.Tensor:
    """float32 [max_positions, rope_dim]: cos of the rotation angles of each position in the first half of a row,
    sin in the second (angle of pair j at position t: t * base ** (-2 j / rope_dim), formed in 64 bits)."""
    if rope_dim < 2 or rope_dim % 2 != 0 or max_positions < 1:
        raise ValueError("rope_dim must be even and positive, max_positions positive")
    dev = device or "cuda"
    freq = base ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=dev) / rope_dim)
    angle = torch.arange(max_positions, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=-1).float().contiguous()


def _need_rows(t, name: str, cols: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype not in _DTYPE:
        raise TypeError(f"{name} must be a bfloat16, float16 or float32 CUDA tensor")
    if t.dim() != 2 or t.shape[1] != cols or t.stride(1) != 1 or (t.shape[0] > 1 and t.stride(0) < cols):
        raise ValueError(f"{name} must be [T,{cols}] with unit stride in a row and rows that do not overlap")


def _need_weight(t, name: str, dtype):
    """A vector of dtype or float32."""
    _need(t, name, torch.float32 if isinstance(t, torch.Tensor) and t.dtype == torch.float32 else dtype, 1)


def _need_paged(kv_cache, block_table, positions, requests, T: int):
    _need(block_table, "block_table", torch.int32, 2)
    _need(positions, "positions", torch.int32, 1)
    _need(kv_cache, "kv_cache", torch.uint8, 3)
    if kv_cache.shape[1] != PAGE_SIZE or kv_cache.shape[2] != 656:
        raise ValueError("kv_cache must be [pages,64,656]")
    if positions.shape[0] != T:
        raise ValueError("positions must be [T]")
    if requests is not None:
        _need(requests, "requests", torch.int32, 1)
        if requests.shape[0] != T:
            raise ValueError("requests must be [T]")
    _same_device(kv_cache.device, block_table=block_table, positions=positions, requests=requests)


def sparse_mla_kv_norm_append(latent: torch.Tensor, rope: torch.Tensor, norm_weight: torch.Tensor, eps: float,
                              cos_sin: torch.Tensor, block_table: torch.Tensor, positions: torch.Tensor,
                              kv_cache: torch.Tensor, requests: Optional[torch.Tensor] = None,
                              interleaved: bool = True, err_word: Optional[torch.Tensor] = None,
                              stream=None) -> None:
    """RMS norm of the latent [T,512] (weight [512]), rotation of the rope [T,64] at its position, FP8
    quantisation and the record write of sparse_mla_kv_append in one pass; kv_cache is written in place.

    latent and rope: bf16, fp16 or fp32, rows may be strided (slices of one projection output); norm_weight of
    their type or fp32; cos_sin fp32 [positions,64] (rope_table)."""
    key = _call_key((latent, rope, norm_weight, cos_sin, block_table, positions, kv_cache, requests, err_word),
                    "kv_norm_append", bool(interleaved))
    dims = _CHECKED.get(key) or _remember(key, _norm_append_dims(latent, rope, norm_weight, cos_sin, block_table,
                                                                 positions, kv_cache, requests, interleaved, err_word))
    with _on(kv_cache.device, stream) as st:
        r = _lib().sparse_mla_kv_norm_append(
            dims, latent.data_ptr(), rope.data_ptr(), norm_weight.data_ptr(), eps, cos_sin.data_ptr(),
            block_table.data_ptr(), _ptr(requests), positions.data_ptr(), kv_cache.data_ptr(), _ptr(err_word), st)
    if r != 0:
        check("sparse_mla_kv_norm_append", r)


def _norm_append_dims(latent, rope, norm_weight, cos_sin, block_table, positions, kv_cache, requests, interleaved,
                      err_word) -> SmlaNormAppendDims:
    _need_rows(latent, "latent", D_LATENT)
    _need_rows(rope, "rope", D_ROPE)
    T = latent.shape[0]
    if rope.shape[0] != T or rope.dtype != latent.dtype:
        raise ValueError("latent and rope need the same number of rows and one type")
    _need_weight(norm_weight, "norm_weight", latent.dtype)
    if norm_weight.shape[0] != D_LATENT:
        raise ValueError("norm_weight must be [512]")
    _need(cos_sin, "cos_sin", torch.float32, 2)
    if cos_sin.shape[1] != D_ROPE:
        raise ValueError("cos_sin must be [positions,64]")
    _need_paged(kv_cache, block_table, positions, requests, T)
    dev = kv_cache.device
    _same_device(dev, latent=latent, rope=rope, norm_weight=norm_weight, cos_sin=cos_sin)
    _err_word(err_word, dev)
    return SmlaNormAppendDims(T, block_table.shape[0], PAGE_SIZE, block_table.shape[1], D_LATENT, D_ROPE,
                              kv_cache.shape[0], latent.stride(0) if T > 1 else D_LATENT,
                              rope.stride(0) if T > 1 else D_ROPE, _DTYPE[latent.dtype], _DTYPE[norm_weight.dtype],
                              cos_sin.shape[0], 1 if interleaved else 0)


def _apart(x: torch.Tensor, out: torch.Tensor, x_bytes: int, out_bytes: int) -> bool:
    """Whether out may be written while x is read: x itself, memory of its own, or other columns of x's rows.  (x_bytes,
    out_bytes: from their first element to their last.)"""
    a, b = x.data_ptr(), out.data_ptr()
    if a + x_bytes <= b or b + out_bytes <= a or (a == b and x.stride() == out.stride()) or x.numel() == 0:
        return True
    # a dim of size 1 may have any stride
    steps = [(s, t) for n, s, t in zip(x.shape[:2], x.stride(), out.stride()) if n > 1]
    if any(s != t for s, t in steps):
        return False
    if a == b:
        return True
    strides = [s for s, _ in steps]
    if not strides or min(strides) < 1 or max(strides) % min(strides) != 0:
        return False
    size, step = x.element_size(), min(strides)
    return size * x.shape[2] <= (b - a) % (size * step) <= size * (step - x.shape[2])


def _span_bytes(t: torch.Tensor) -> int:
    return t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))


def sparse_mla_norm_rope(x: torch.Tensor, positions: Optional[torch.Tensor] = None,
                         cos_sin: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                         eps: float = 1e-6, norm: bool = True, rope_offset: int = 0, interleaved: bool = True,
                         out: Optional[torch.Tensor] = None, err_word: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """x [T,H,D] (bf16, fp16 or fp32, unit stride along D): RMS norm of each head's vector (norm, with an optional
    weight [D] of x's type or fp32), then rotation of the dims [rope_offset, rope_offset + cos_sin.shape[1]) at
    positions [T] (cos_sin fp32, rope_table; None: no rotation).  out: as x, or x itself."""
    key = _call_key((x, positions, cos_sin, weight, out, err_word), "norm_rope", bool(norm), rope_offset, bool(interleaved))
    dims, x_bytes, out_bytes = _CHECKED.get(key) or _remember(
        key, _norm_rope_dims(x, positions, cos_sin, weight, norm, rope_offset, interleaved, out, err_word))
    with _on(x.device, stream) as st:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        elif not _apart(x, out, x_bytes, out_bytes):
            raise ValueError("out must be x itself or not overlap it")
        r = _lib().sparse_mla_norm_rope(
            dims, x.data_ptr(), _ptr(weight), eps, _ptr(cos_sin), positions.data_ptr() if dims.rope_dim else None,
            out.data_ptr(), _ptr(err_word), st)
    if r != 0:
        check("sparse_mla_norm_rope", r)
    return out


def _norm_rope_dims(x, positions, cos_sin, weight, norm, rope_offset, interleaved, out, err_word):
    """Checked dims, and the bytes that x and out span."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if not x.is_cuda or x.dtype not in _DTYPE:
        raise TypeError("x must be a bfloat16, float16 or float32 CUDA tensor")
    if x.dim() != 3 or x.shape[1] < 1 or x.shape[2] < 1 or (x.shape[2] > 1 and x.stride(2) != 1):
        raise ValueError("x must be [T,H,D] with unit stride along D")
    T, H, D = x.shape
    if weight is not None:
        if not norm:
            raise ValueError("weight without norm")
        _need_weight(weight, "weight", x.dtype)
        if weight.shape[0] != D:
            raise ValueError("weight must be [D]")
    rope_dim = max_pos = 0
    if cos_sin is not None:
        _need(cos_sin, "cos_sin", torch.float32, 2)
        if positions is None:
            raise ValueError("cos_sin without positions")
        _need(positions, "positions", torch.int32, 1)
        if positions.shape[0] != T:
            raise ValueError("positions must be [T]")
        max_pos, rope_dim = cos_sin.shape
    _same_device(x.device, weight=weight, cos_sin=cos_sin, positions=positions, out=out)
    _err_word(err_word, x.device)
    if out is not None and (out.shape != x.shape or out.dtype != x.dtype or (D > 1 and out.stride(2) != 1)):
        raise ValueError("out must have x's shape and type and unit stride along D")
    o_strides = (H * D, D) if out is None else out.stride()
    dims = SmlaNormRopeDims(T, H, D, rope_dim, rope_offset, _DTYPE[x.dtype],
                            _DTYPE[weight.dtype if weight is not None else x.dtype], 1 if norm else 0,
                            1 if interleaved else 0, max_pos, x.stride(0), x.stride(1), o_strides[0], o_strides[1])
    return dims, _span_bytes(x), 0 if out is None else _span_bytes(out)


def sparse_mla_kv_read(kv_cache: torch.Tensor, block_table: torch.Tensor, positions: torch.Tensor,
                       requests: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       dtype: torch.dtype = torch.bfloat16, err_word: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """[T,576]: the records at (requests[i] or i, positions[i]) as [latent * scale | rope] rows of dtype (out's type
    when out is given); zeros for a token out of range."""
    key = _call_key((kv_cache, block_table, positions, requests, out, err_word), "kv_read", dtype)
    dims, dtype = _CHECKED.get(key) or _remember(key, _read_dims(kv_cache, block_table, positions, requests, out, dtype,
                                                                 err_word))
    with _on(kv_cache.device, stream) as st:
        if out is None:
            out = torch.empty((positions.shape[0], D_QK), dtype=dtype, device=kv_cache.device)
        r = _lib().sparse_mla_kv_read(dims, kv_cache.data_ptr(), block_table.data_ptr(), _ptr(requests),
                                      positions.data_ptr(), out.data_ptr(), _DTYPE[dtype], _ptr(err_word), st)
    if r != 0:
        check("sparse_mla_kv_read", r)
    return out


def _read_dims(kv_cache, block_table, positions, requests, out, dtype, err_word):
    """Checked dims and the output's type."""
    T = positions.shape[0] if isinstance(positions, torch.Tensor) and positions.dim() == 1 else -1
    _need_paged(kv_cache, block_table, positions, requests, T)
    dev = kv_cache.device
    if out is not None:
        dtype = out.dtype
        _need(out, "out", dtype, 2)
        if out.shape != (T, D_QK) or out.device != dev:
            raise ValueError(f"out must be [T,576] on {dev}")
    if dtype not in _DTYPE:
        raise TypeError("out must be bfloat16, float16 or float32")
    _err_word(err_word, dev)
    return SmlaAppendDims(T, block_table.shape[0], PAGE_SIZE, block_table.shape[1], D_LATENT, D_ROPE,
                          kv_cache.shape[0]), dtype


def make_dense_dims(B: int, H: int, max_pages_per_seq: int, num_pages: int, queries_per_request: int = 1,
                    ctas: int = 0) -> SmlaDenseDims:
    return SmlaDenseDims(B, H, PAGE_SIZE, max_pages_per_seq, D_LATENT, D_ROPE, num_pages, queries_per_request, ctas)


def dense_dims_of(q, kv_cache, block_table, ctas: int = 0) -> SmlaDenseDims:
    """Shapes of a dense decode; several queries per request when q has a multiple of block_table's rows."""
    return make_dense_dims(q.shape[0], q.shape[1], block_table.shape[1], kv_cache.shape[0],
                           q.shape[0] // block_table.shape[0], ctas)


def dense_plan_for(dims: SmlaDenseDims, sm_count: int) -> SmlaDensePlan:
    p = SmlaDensePlan()
    check("sparse_mla_dense_plan_for", _lib().sparse_mla_dense_plan_for(C.byref(dims), sm_count, C.byref(p)))
    return p


def dense_plan(dims: SmlaDenseDims, device: Optional[int] = None) -> SmlaDensePlan:
    p = SmlaDensePlan()
    dev = torch.cuda.current_device() if device is None else device
    check("sparse_mla_dense_plan", _lib().sparse_mla_dense_plan(C.byref(dims), dev, C.byref(p)))
    return p


def alloc_dense_workspace(dims: SmlaDenseDims, device=None) -> torch.Tensor:
    """Caller-owned workspace of sparse_mla_dense_decode with a clear error word."""
    dev = torch.device(device or "cuda")
    ws = torch.empty(dense_plan(dims, dev.index).workspace_bytes, dtype=torch.uint8, device=dev)
    ws[:256].zero_()
    return ws


# Dense decode dims by call shape (the library reads dims, never writes them).
_DENSE_DIMS = {}


def sparse_mla_dense_decode(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                            seq_lens: torch.Tensor, sm_scale: float, out: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            stream=None, ctas: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of q bf16 [B,H,576] over every position below seq_lens[b] of its request's cache: out bf16
    [B,H,512], lse fp32 [B,H].  H is 1 .. 128; block_table has one row per request, seq_lens one entry per query
    (B a multiple of the requests).  ctas = 0: one CTA per SM.  Calls in flight at once need a workspace each
    (alloc_dense_workspace); without one a call allocates its own, and its error word is lost."""
    _need(q, "q", torch.bfloat16, 3)
    _need(kv_cache, "kv_cache", torch.uint8, 3)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    dev = q.device
    key = (q.shape, kv_cache.shape, block_table.shape, seq_lens.shape, ctas)
    dims = _DENSE_DIMS.get(key)
    if dims is None:
        B, R = q.shape[0], block_table.shape[0]
        if q.shape[2] != D_QK or kv_cache.shape[1] != PAGE_SIZE or kv_cache.shape[2] != 656:
            raise ValueError("q must be [B,H,576] and kv_cache [pages,64,656]")
        if R < 1 or B % R != 0 or seq_lens.shape[0] != B:
            raise ValueError("q and seq_lens need one row per query, block_table one row per request (a divisor of "
                             "the query count)")
        dims = dense_dims_of(q, kv_cache, block_table, ctas)
        if len(_DENSE_DIMS) > 256:
            _DENSE_DIMS.clear()
        _DENSE_DIMS[key] = dims
    _same_device(dev, kv_cache=kv_cache, block_table=block_table, seq_lens=seq_lens, out=out, lse=lse,
                 workspace=workspace)
    with _on(dev, stream) as st:
        if out is None:
            out = torch.empty((q.shape[0], q.shape[1], D_LATENT), dtype=torch.bfloat16, device=dev)
        else:
            _need(out, "out", torch.bfloat16, 3)
            if out.shape[:2] != q.shape[:2] or out.shape[2] != D_LATENT:
                raise ValueError("out must be [B,H,512]")
        if lse is None:
            lse = torch.empty((q.shape[0], q.shape[1]), dtype=torch.float32, device=dev)
        else:
            _need(lse, "lse", torch.float32, 2)
            if lse.shape != q.shape[:2]:
                raise ValueError("lse must be [B,H]")
        if workspace is None:
            workspace = alloc_dense_workspace(dims, dev)
        else:
            _need(workspace, "workspace", torch.uint8, 1)
        r = _lib().sparse_mla_dense_decode(
            dims, q.data_ptr(), kv_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), sm_scale,
            out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(), st)
    if r != 0:
        check("sparse_mla_dense_decode", r)
    return out, lse


def sparse_mla_topk_select(scores: torch.Tensor, seq_lens: torch.Tensor, k: int, cluster_ctas: int = 0,
                           err_word: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """int32 [B,k]: per query the k positions below seq_lens[b] of largest score (IEEE totalOrder,
    ties to the lower position), in increasing order, -1 padded when seq_lens[b] <= k.
    scores float32 [B, num_cols] with unit stride along positions."""
    _need(seq_lens, "seq_lens", torch.int32, 1)
    if scores.dtype != torch.float32 or scores.dim() != 2 or not scores.is_cuda:
        raise ValueError("scores must be a float32 [B, num_cols] CUDA tensor")
    if scores.stride(1) != 1 or (scores.shape[0] > 1 and scores.stride(0) < scores.shape[1]):
        raise ValueError("scores rows must be contiguous")
    B, n = scores.shape
    if seq_lens.shape[0] != B:
        raise ValueError("seq_lens must be [B]")
    out = torch.empty((B, k), dtype=torch.int32, device=scores.device)
    dims = SmlaTopkDims(B, n, scores.stride(0) if B > 1 else n, k, cluster_ctas)
    check("sparse_mla_topk_select", _lib().sparse_mla_topk_select(
        C.byref(dims), _ptr(scores), _ptr(seq_lens), _ptr(out), _ptr(err_word), _stream(stream)))
    return out


def sparse_mla_combine(o_part: torch.Tensor, lse_part: torch.Tensor, stream=None):
    _need(o_part, "o_part", torch.float32, 4)
    _need(lse_part, "lse_part", torch.float32, 3)
    B, S, H, D = o_part.shape
    out = torch.empty((B, H, D), dtype=torch.bfloat16, device=o_part.device)
    lse = torch.empty((B, H), dtype=torch.float32, device=o_part.device)
    check("sparse_mla_combine", _lib().sparse_mla_combine(B, H, S, _ptr(o_part), _ptr(lse_part), _ptr(out),
                                                          _ptr(lse), _stream(stream)))
    return out, lse


def sparse_mla_gather_rows(block_table, topk_idx, seq_lens, num_pages: int, stream=None) -> torch.Tensor:
    _need(block_table, "block_table", torch.int32, 2)
    _need(topk_idx, "topk_idx", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, K = topk_idx.shape
    if block_table.shape[0] < 1 or B % block_table.shape[0] != 0:
        raise ValueError("block_table needs one row per request (a divisor of the query count)")
    dims = make_dims(B, 64, K, block_table.shape[1], num_pages, queries_per_request=B // block_table.shape[0])
    rows = torch.empty((B, K), dtype=torch.int64, device=topk_idx.device)
    check("sparse_mla_gather_rows", _lib().sparse_mla_gather_rows(
        C.byref(dims), _ptr(block_table), _ptr(topk_idx), _ptr(seq_lens), _ptr(rows), _stream(stream)))
    return rows


def clear_errors(workspace: torch.Tensor, stream=None) -> None:
    check("sparse_mla_clear_errors", _lib().sparse_mla_clear_errors(_ptr(workspace), _stream(stream)))


def read_errors(workspace: torch.Tensor, stream=None) -> int:
    v = C.c_uint32(0)
    check("sparse_mla_read_errors", _lib().sparse_mla_read_errors(_ptr(workspace), C.byref(v), _stream(stream)))
    return int(v.value)
