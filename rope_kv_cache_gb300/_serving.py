"""Binding of libropekv_serving.so (include/ropekv_serving.h): rotary positions
with several axes, the 8-bit cache with a scale per token and head, reading a
paged cache back, and shared-prefix attention.

As the functions of ``_binding``: torch CUDA tensors in the header's layouts,
checks of type, device, layout and shape, one call of the C entry point on the
current (or given) stream, RopeKVError for a non-zero status, no fallback. The
checks and the call are in a compiled module (csrc/ropekv_bind.cpp).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional, Sequence

import torch

from ._binding import NEOX, RopeKVError
from .build import bind_path

_LIB_DIR = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib")
SERVING_LIB_PATH = os.path.join(_LIB_DIR, "libropekv_serving.so")
_lib = None
_bind = None


class ropekv_attention_dims(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in (
        "batch", "seqLen", "numQHeads", "numKVHeads", "headDim", "numPages", "tokensPerPage",
        "maxPagesPerSeq", "prefixLen", "maxPrefixPages", "cacheFormat")]


def _require(path: str) -> str:
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built; run `python -c \"import __graft_entry__ as g; g.build()\"` "
            "(needs nvcc) -- there is no CPU fallback")
    return path


def _native():
    """The compiled binding of the running torch, loaded once."""
    global _bind
    if _bind is None:
        _require(SERVING_LIB_PATH)
        spec = importlib.util.spec_from_file_location("ropekv_bind", _require(bind_path()))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _bind = module
    return _bind


def load_serving_library():
    """libropekv_serving.so itself, by ctypes, loaded once: the C entry points as the header
    declares them."""
    global _lib
    if _lib is None:
        _require(SERVING_LIB_PATH)
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
    rc = (_bind or _native()).mrope(cos_sin, positions, freq_axis, q, k, v, slot_mapping, key_cache,
                                    value_cache, q_out, k_out, style, stream)
    if rc:
        raise RopeKVError("rope_write_kv_mrope", rc)


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
    rc = (_bind or _native()).quant(cos_sin, positions, q, k, v, slot_mapping, key_cache, value_cache,
                                    key_scales, value_scales, q_out, style, stream)
    if rc:
        raise RopeKVError("rope_write_kv_slot_mapping_quant", rc)


def paged_kv_read(kv_cache: torch.Tensor, page_table: torch.Tensor, row_positions: torch.Tensor,
                  row_sequences: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor,
                  kv_scales: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Rows of a paged cache as dense FP16: row t of k_out, v_out [N, Hkv, D] float16 takes
    position row_positions[t] of sequence row_sequences[t] ([N] int32). kv_cache
    [2, P, TPP, Hkv, D] float16, float8_e4m3fn or int8 (the 8-bit ones with kv_scales
    [2, P, Hkv, TPP] float32); page_table [B, 2, M] int32. Skipped rows keep their
    contents."""
    rc = (_bind or _native()).read(kv_cache, page_table, row_positions, row_sequences, k_out, v_out,
                                   kv_scales, stream)
    if rc:
        raise RopeKVError("paged_kv_read", rc)


def paged_attention_workspace_size(q: torch.Tensor, kv_cache: torch.Tensor,
                                   prefix_table: Optional[torch.Tensor], prefix_len: int,
                                   page_table: torch.Tensor,
                                   kv_scales: Optional[torch.Tensor] = None) -> int:
    """Bytes of workspace that paged_attention_shared_prefix needs for these tensors."""
    n = (_bind or _native()).attention_workspace(q, kv_cache, prefix_table, prefix_len, page_table,
                                                 kv_scales)
    if n < 0:
        raise RopeKVError("paged_attention_workspace_size", n)
    return n


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
    rc = (_bind or _native()).attention(q, kv_cache, prefix_table, prefix_len, page_table, kv_lens, out,
                                        lse, kv_scales, sm_scale, workspace, stream)
    if rc:
        raise RopeKVError("paged_attention_shared_prefix", rc)
