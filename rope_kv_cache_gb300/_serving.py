"""ctypes binding of libropekv_serving.so (include/ropekv_serving.h): rotary
positions with several axes, the 8-bit cache with a scale per token and head,
reading a paged cache back, and shared-prefix attention.

As the functions of ``_binding``: torch CUDA tensors in the header's layouts,
checks of type, device, layout and shape, one call of the C entry point on the
current (or given) stream, RopeKVError for a non-zero status, no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import torch

from ._binding import NEOX, RopeKVError

CACHE_F16, CACHE_E4M3, CACHE_INT8 = 0, 1, 2
_FORMATS = {torch.float16: CACHE_F16, torch.float8_e4m3fn: CACHE_E4M3, torch.int8: CACHE_INT8}

SERVING_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib",
                                "libropekv_serving.so")
_lib = None


class ropekv_attention_dims(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in (
        "batch", "seqLen", "numQHeads", "numKVHeads", "headDim", "numPages", "tokensPerPage",
        "maxPagesPerSeq", "prefixLen", "maxPrefixPages", "cacheFormat")]


def load_serving_library():
    """Load libropekv_serving.so once. Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(SERVING_LIB_PATH):
            raise RuntimeError(
                f"{SERVING_LIB_PATH} is not built; run `python -c \"import __graft_entry__ as g; "
                "g.build()\"` (needs nvcc) -- there is no CPU fallback")
        lib = ctypes.CDLL(SERVING_LIB_PATH)
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        D = ctypes.POINTER(ropekv_attention_dims)
        lib.rope_write_kv_mrope.argtypes = [P, P, P, I32, P, I64, P, I64, P, I64, P, P, P, P, P,
                                            I32, I32, I32, I32, I32, I32, I64, I32, I32, P]
        lib.rope_write_kv_slot_mapping_quant.argtypes = [P, P, P, I64, P, I64, P, I64, P, P, P, P,
                                                         P, P, I32, I32, I32, I32, I32, I32, I64,
                                                         I32, I32, I32, P]
        lib.paged_kv_read.argtypes = [P] * 7 + [I32] * 8 + [P]
        lib.paged_attention_workspace_size.argtypes = [D]
        lib.paged_attention_workspace_size.restype = I64
        lib.paged_attention_shared_prefix.argtypes = [P] * 9 + [I64, D, ctypes.c_float, P]
        for fn in ("rope_write_kv_mrope", "rope_write_kv_slot_mapping_quant", "paged_kv_read",
                   "paged_attention_shared_prefix"):
            getattr(lib, fn).restype = ctypes.c_int
        _lib = lib
    return _lib


# ------------------------------------------------------------- marshalling --

def _on(t: torch.Tensor, name: str, device) -> None:
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name} is on {t.device}, expected " +
                         (str(device) if device.type == "cuda" else "a CUDA device"))


def _ptr(t: Optional[torch.Tensor], name: str, dtype, device) -> Optional[int]:
    """Address of a dense CUDA tensor of `dtype` on `device`; None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    _on(t, name, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, device):
    """Address and token stride of a [T, H, D] float16 tensor with dense heads and dims."""
    if t.dtype != torch.float16:
        raise TypeError(f"{name}: dtype {t.dtype}, expected torch.float16")
    _on(t, name, device)
    T, H, D = t.shape
    st = t.stride()
    if st[2] != 1 or (H > 1 and st[1] != D):
        raise ValueError(f"{name}: heads and dims must be dense (strides (*, D, 1))")
    return t.data_ptr(), (st[0] if T > 1 else H * D)


def _format(t: torch.Tensor, name: str, eight_bit_only: bool = False) -> int:
    fmt = _FORMATS.get(t.dtype)
    if fmt is None or (eight_bit_only and fmt == CACHE_F16):
        raise TypeError(f"{name}: dtype {t.dtype}, expected " +
                        ("" if eight_bit_only else "float16, ") + "float8_e4m3fn or int8")
    return fmt


def _launch(fn: str, device, stream, *args) -> None:
    """Call the entry point with the tensors' device current and the stream last."""
    f = getattr(_lib or load_serving_library(), fn)
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if torch.cuda.current_device() == device.index:
        rc = f(*args, stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            rc = f(*args, stream.cuda_stream)
    if rc != 0:
        raise RopeKVError(fn, rc)


def _check_write(fn, cos_sin, positions_shape, positions, q, k, v, slot_mapping, key_cache,
                 value_cache, q_out):
    if q.dim() != 3 or k.dim() != 3 or key_cache.dim() != 4 or cos_sin.dim() != 2:
        raise ValueError("cos_sin [rows,r], q [T,Hq,D], k [T,Hkv,D], key_cache "
                         "[blocks,block_size,Hkv,D] expected")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (T, Hkv, D) or tuple(v.shape) != (T, Hkv, D) \
            or tuple(positions.shape) != positions_shape or tuple(slot_mapping.shape) != (T,) \
            or tuple(key_cache.shape[2:]) != (Hkv, D) or value_cache.shape != key_cache.shape \
            or tuple(q_out.shape) != (T, Hq, D):
        raise ValueError(f"inconsistent shapes for {fn}")
    return T, Hq, Hkv, D


# ------------------------------------------------------------ entry points --

def mrope_freq_axis(sections: Sequence[int], interleaved: bool = False) -> torch.Tensor:
    """Axis of each frequency for ``rope_write_kv_mrope`` (int32 CPU tensor).

    sections[a] frequencies belong to axis a, sum(sections) = rotaryDim / 2.
    Chunked (default): the first sections[0] frequencies take axis 0, the next
    sections[1] axis 1, and so on. Interleaved: axis a > 0 takes frequencies a,
    a + A, a + 2A, ... (A axes), axis 0 all others."""
    axes, n = len(sections), sum(sections)
    if axes < 1 or axes > 4 or min(sections) < 0:
        raise ValueError("1 to 4 sections, none negative, expected")
    if not interleaved:
        return torch.tensor([a for a, s in enumerate(sections) for _ in range(s)], dtype=torch.int32)
    out = [0] * n
    for a in range(1, axes):
        for j in range(sections[a]):
            f = a + j * axes
            if f >= n:
                raise ValueError(f"axis {a}: {sections[a]} interleaved frequencies do not fit in {n}")
            out[f] = a
    return torch.tensor(out, dtype=torch.int32)


def rope_write_kv_mrope(cos_sin: torch.Tensor, positions: torch.Tensor, freq_axis: torch.Tensor,
                        q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        slot_mapping: torch.Tensor, key_cache: torch.Tensor,
                        value_cache: torch.Tensor, q_out: torch.Tensor,
                        k_out: Optional[torch.Tensor] = None, style: int = NEOX,
                        stream: Optional[torch.cuda.Stream] = None) -> None:
    """rope_write_kv_slot_mapping with several position axes: frequency i of token t
    takes the cos/sin row positions[freq_axis[i], t].

    cos_sin [rows, r] float32; positions [axes, T] int64; freq_axis [r/2] int32 on the
    CPU (see ``mrope_freq_axis``); the others as rope_write_kv_slot_mapping."""
    if positions.dim() != 2:
        raise ValueError("positions [axes, T] expected")
    axes = positions.shape[0]
    T, Hq, Hkv, D = _check_write("rope_write_kv_mrope", cos_sin, (axes, q.shape[0]), positions, q, k,
                                 v, slot_mapping, key_cache, value_cache, q_out)
    r = cos_sin.shape[1]
    if k_out is not None and tuple(k_out.shape) != (T, Hkv, D):
        raise ValueError("k_out [T, Hkv, D] expected")
    if freq_axis.dtype != torch.int32 or freq_axis.device.type != "cpu" \
            or tuple(freq_axis.shape) != (r // 2,) or not freq_axis.is_contiguous():
        raise ValueError("freq_axis must be a contiguous int32 CPU tensor of r/2 elements")
    dev = q.device
    qp, qs = _rows(q, "q", dev)
    kp, ks = _rows(k, "k", dev)
    vp, vs = _rows(v, "v", dev)
    f16, i64 = torch.float16, torch.int64
    _launch("rope_write_kv_mrope", dev, stream, _ptr(cos_sin, "cos_sin", torch.float32, dev),
            _ptr(positions, "positions", i64, dev), freq_axis.data_ptr(), axes, qp, qs, kp, ks, vp,
            vs, _ptr(slot_mapping, "slot_mapping", i64, dev), _ptr(key_cache, "key_cache", f16, dev),
            _ptr(value_cache, "value_cache", f16, dev), _ptr(q_out, "q_out", f16, dev),
            _ptr(k_out, "k_out", f16, dev), T, Hq, Hkv, D, r, cos_sin.shape[0], key_cache.shape[0],
            key_cache.shape[1], style)


def rope_write_kv_slot_mapping_quant(cos_sin: torch.Tensor, positions: torch.Tensor,
                                     q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                     slot_mapping: torch.Tensor, key_cache: torch.Tensor,
                                     value_cache: torch.Tensor, key_scales: torch.Tensor,
                                     value_scales: torch.Tensor, q_out: torch.Tensor,
                                     style: int = NEOX,
                                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """rope_write_kv_slot_mapping into an 8-bit cache: key_cache, value_cache
    [blocks, block_size, Hkv, D] float8_e4m3fn or int8, key_scales, value_scales
    [blocks, Hkv, block_size] float32, one scale per token and KV head, found as the
    token is written."""
    T, Hq, Hkv, D = _check_write("rope_write_kv_slot_mapping_quant", cos_sin, (q.shape[0],),
                                 positions, q, k, v, slot_mapping, key_cache, value_cache, q_out)
    blocks, bs = key_cache.shape[:2]
    if tuple(key_scales.shape) != (blocks, Hkv, bs) or key_scales.shape != value_scales.shape:
        raise ValueError("key_scales, value_scales [blocks, Hkv, block_size] expected")
    fmt = _format(key_cache, "key_cache", eight_bit_only=True)
    dev = q.device
    qp, qs = _rows(q, "q", dev)
    kp, ks = _rows(k, "k", dev)
    vp, vs = _rows(v, "v", dev)
    f32, i64 = torch.float32, torch.int64
    _launch("rope_write_kv_slot_mapping_quant", dev, stream, _ptr(cos_sin, "cos_sin", f32, dev),
            _ptr(positions, "positions", i64, dev), qp, qs, kp, ks, vp, vs,
            _ptr(slot_mapping, "slot_mapping", i64, dev),
            _ptr(key_cache, "key_cache", key_cache.dtype, dev),
            _ptr(value_cache, "value_cache", key_cache.dtype, dev),
            _ptr(key_scales, "key_scales", f32, dev), _ptr(value_scales, "value_scales", f32, dev),
            _ptr(q_out, "q_out", torch.float16, dev), T, Hq, Hkv, D, cos_sin.shape[1],
            cos_sin.shape[0], blocks, bs, fmt, style)


def _check_pool(kv_cache, kv_scales, page_table):
    """Sizes of a paged pool, its scales and a page table: (P, tpp, Hkv, D, fmt, B, M)."""
    if kv_cache.dim() != 5 or kv_cache.shape[0] != 2 or page_table.dim() != 3 \
            or page_table.shape[1] != 2:
        raise ValueError("kv_cache [2,P,TPP,Hkv,D] and page_table [B,2,M] expected")
    _, pages, tpp, Hkv, D = kv_cache.shape
    fmt = _format(kv_cache, "kv_cache")
    if fmt == CACHE_F16:
        if kv_scales is not None:
            raise ValueError("a float16 cache has no kv_scales")
    elif kv_scales is None or tuple(kv_scales.shape) != (2, pages, Hkv, tpp):
        raise ValueError("kv_scales [2, P, Hkv, TPP] expected for an 8-bit cache")
    return pages, tpp, Hkv, D, fmt, page_table.shape[0], page_table.shape[2]


def paged_kv_read(kv_cache: torch.Tensor, page_table: torch.Tensor, row_positions: torch.Tensor,
                  row_sequences: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor,
                  kv_scales: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Rows of a paged cache as dense FP16: row t of k_out, v_out [N, Hkv, D] float16 takes
    position row_positions[t] of sequence row_sequences[t] ([N] int32). kv_cache
    [2, P, TPP, Hkv, D] float16, float8_e4m3fn or int8 (the 8-bit ones with kv_scales
    [2, P, Hkv, TPP] float32); page_table [B, 2, M] int32. Skipped rows keep their
    contents."""
    pages, tpp, Hkv, D, fmt, B, M = _check_pool(kv_cache, kv_scales, page_table)
    if row_positions.dim() != 1 or row_sequences.shape != row_positions.shape \
            or tuple(k_out.shape) != (row_positions.shape[0], Hkv, D) or v_out.shape != k_out.shape:
        raise ValueError("row_positions, row_sequences [N] and k_out, v_out [N, Hkv, D] expected")
    dev, i32, f16 = kv_cache.device, torch.int32, torch.float16
    _launch("paged_kv_read", dev, stream, _ptr(kv_cache, "kv_cache", kv_cache.dtype, dev),
            _ptr(kv_scales, "kv_scales", torch.float32, dev), _ptr(page_table, "page_table", i32, dev),
            _ptr(row_positions, "row_positions", i32, dev),
            _ptr(row_sequences, "row_sequences", i32, dev), _ptr(k_out, "k_out", f16, dev),
            _ptr(v_out, "v_out", f16, dev), row_positions.shape[0], B, Hkv, D, pages, M, tpp, fmt)


def _attention_dims(q, kv_cache, kv_scales, prefix_table, prefix_len, page_table):
    if q.dim() != 4:
        raise ValueError("q [B, S, Hq, D] expected")
    pages, tpp, Hkv, D, fmt, B, M = _check_pool(kv_cache, kv_scales, page_table)
    if q.shape[0] != B or q.shape[3] != D:
        raise ValueError(f"q {tuple(q.shape)} does not match page_table {tuple(page_table.shape)} "
                         f"and kv_cache {tuple(kv_cache.shape)}")
    if prefix_table is None:
        cols = 0
    elif prefix_table.dim() != 2 or prefix_table.shape[0] != 2:
        raise ValueError("prefix_table [2, prefix pages] expected")
    else:
        cols = prefix_table.shape[1]
    return ropekv_attention_dims(B, q.shape[1], q.shape[2], Hkv, D, pages, tpp, M, int(prefix_len),
                                 cols, fmt)


def _workspace_size(dims) -> int:
    n = (_lib or load_serving_library()).paged_attention_workspace_size(ctypes.byref(dims))
    if n < 0:
        raise RopeKVError("paged_attention_workspace_size", int(n))
    return n


def paged_attention_workspace_size(q: torch.Tensor, kv_cache: torch.Tensor,
                                   prefix_table: Optional[torch.Tensor], prefix_len: int,
                                   page_table: torch.Tensor,
                                   kv_scales: Optional[torch.Tensor] = None) -> int:
    """Bytes of workspace that paged_attention_shared_prefix needs for these tensors."""
    return _workspace_size(_attention_dims(q, kv_cache, kv_scales, prefix_table, prefix_len,
                                           page_table))


def paged_attention_shared_prefix(q: torch.Tensor, kv_cache: torch.Tensor,
                                  prefix_table: Optional[torch.Tensor], prefix_len: int,
                                  page_table: torch.Tensor, kv_lens: torch.Tensor,
                                  out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                                  kv_scales: Optional[torch.Tensor] = None,
                                  sm_scale: Optional[float] = None,
                                  workspace: Optional[torch.Tensor] = None,
                                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Attention of S new tokens per sequence over a paged cache whose first prefix_len
    positions all sequences share.

    q, out [B, S, Hq, D] float16; kv_cache [2, P, TPP, Hkv, D] float16, float8_e4m3fn or int8
    (8-bit ones with kv_scales [2, P, Hkv, TPP] float32); prefix_table [2, prefix pages] int32
    (None when prefix_len is 0); page_table [B, 2, M] int32; kv_lens [B] int32, lengths with
    the prefix and the new tokens; lse [B, S, Hq] float32 or None; sm_scale defaults to
    D^-0.5. workspace: a uint8 tensor of paged_attention_workspace_size bytes, or None: one
    is allocated for the call on the stream it runs on."""
    dims = _attention_dims(q, kv_cache, kv_scales, prefix_table, prefix_len, page_table)
    if tuple(kv_lens.shape) != (dims.batch,) or out.shape != q.shape \
            or (lse is not None and lse.shape != q.shape[:3]):
        raise ValueError("kv_lens [B], out [B,S,Hq,D], lse [B,S,Hq] expected")
    dev, i32, f16, f32 = q.device, torch.int32, torch.float16, torch.float32
    args = (_ptr(q, "q", f16, dev), _ptr(kv_cache, "kv_cache", kv_cache.dtype, dev),
            _ptr(kv_scales, "kv_scales", f32, dev), _ptr(prefix_table, "prefix_table", i32, dev),
            _ptr(page_table, "page_table", i32, dev), _ptr(kv_lens, "kv_lens", i32, dev),
            _ptr(out, "out", f16, dev), _ptr(lse, "lse", f32, dev))
    if workspace is None:
        need = _workspace_size(dims)
        if need:
            with torch.cuda.stream(stream):  # the allocator orders reuse by this stream
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        size = need
    else:
        size = workspace.numel()
    _launch("paged_attention_shared_prefix", dev, stream, *args,
            _ptr(workspace, "workspace", torch.uint8, dev), size, ctypes.byref(dims),
            float(sm_scale) if sm_scale is not None else 1.0 / math.sqrt(q.shape[3]))
