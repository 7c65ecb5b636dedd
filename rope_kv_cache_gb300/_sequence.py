"""Binding of the operators on whole sequences (libropekv_serving.so,
include/ropekv_sequence.h): attention of packed prompts, attention of new tokens (one, a
chain or a tree of drafts) over the contiguous cache, the rows of accepted drafts moved to
the front, and pages of a paged cache copied, forked and freed.

As ``_serving``: torch CUDA tensors in the header's layouts, checks and the call in the
compiled module, RopeKVError for a non-zero status, no fallback.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import _serving
from ._binding import RopeKVError


def _native():
    return _serving._bind or _serving._native()


def _check(fn: str, rc: int) -> int:
    if rc < 0:
        raise RopeKVError(fn, rc)
    return rc


def prompt_attention_workspace_size(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor,
                                    kv_starts: Optional[torch.Tensor] = None) -> int:
    """Bytes of workspace that prompt_attention needs for these tensors."""
    return _check("prompt_attention_workspace_size", _native().prompt_workspace(q, k, v, q_starts, kv_starts))


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor,
                     out: torch.Tensor, kv_starts: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
                     workspace: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """Causal attention of sequences packed one behind another: query i of sequence b, at row
    q_starts[b] + i, sees the keys 0 .. nk - nq + i of its sequence, which begin at row kv_starts[b].

    q [T, Hq, D], k, v [Tk, Hkv, D] float16, token-strided views allowed; q_starts, kv_starts
    [B + 1] int32 (kv_starts defaults to q_starts); out [T, Hq, D] float16; lse [T, Hq] float32
    or None; sm_scale defaults to D^-0.5. workspace: a uint8 tensor of
    prompt_attention_workspace_size bytes, or None: one is allocated for the call on the stream
    it runs on. Rows of no sequence keep their contents."""
    _check("prompt_attention", _native().prompt(q, k, v, q_starts, out, kv_starts, lse, sm_scale, workspace, stream))


def tree_mask_from_parents(parents: Sequence[Sequence[int]]) -> torch.Tensor:
    """Mask for ``tree_attention`` (int32 CPU tensor [B, S, ceil(S / 32)]): parents[b][i] is the
    number of node i's parent among the new tokens of sequence b, below i, or -1 for a root.
    Every node sees itself and its ancestors."""
    B, S = len(parents), len(parents[0]) if parents else 0
    out = torch.zeros(B, S, (S + 31) // 32, dtype=torch.int32)
    for b, row in enumerate(parents):
        if len(row) != S:
            raise ValueError("every sequence must have the same number of nodes")
        sees = []
        for i, p in enumerate(row):
            if p < -1 or p >= i:
                raise ValueError(f"sequence {b}: parent {p} of node {i} must be -1 or below {i}")
            sees.append((sees[p] if p >= 0 else 0) | 1 << i)
            for w in range(out.shape[2]):
                word = sees[i] >> 32 * w & 0xFFFFFFFF
                out[b, i, w] = word - (1 << 32) if word >> 31 else word
    return out


def tree_attention_workspace_size(q: torch.Tensor, kv_cache: torch.Tensor) -> int:
    """Bytes of workspace that tree_attention needs for these tensors."""
    return _check("tree_attention_workspace_size", _native().tree_workspace(q, kv_cache))


def tree_attention(q: torch.Tensor, kv_cache: torch.Tensor, kv_cache_end_lens: torch.Tensor,
                   out: torch.Tensor, tree_mask: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
                   workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """Attention of S new tokens per sequence over the contiguous cache that
    rope_write_kv_tree or rope_write_kv_continuous wrote: token j of sequence b is at slot
    kv_cache_end_lens[b] - S + j and sees all slots before the new tokens, and of those the ones
    that tree_mask names (without one: itself and those before it).

    q, out [B, S, Hq, D] float16; kv_cache [B, 2, Hkv, cap, D] float16; kv_cache_end_lens [B]
    int32; tree_mask [B, S, ceil(S / 32)] int32 (see ``tree_mask_from_parents``) or None; lse
    [B, S, Hq] float32 or None; sm_scale defaults to D^-0.5; workspace as prompt_attention's."""
    _check("tree_attention", _native().tree(q, kv_cache, kv_cache_end_lens, out, tree_mask, lse, sm_scale,
                                            workspace, stream))


def kv_accept_drafts(kv_cache: torch.Tensor, kv_cache_end_lens: torch.Tensor, seq_len: int,
                     accepted: torch.Tensor, accepted_lens: torch.Tensor,
                     end_lens_out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """Moves the rows of accepted drafts to the front of the seq_len new tokens of the
    contiguous cache [B, 2, Hkv, cap, D] float16: entry j < accepted_lens[b] goes from slot
    kv_cache_end_lens[b] - seq_len + accepted[b, j] to slot kv_cache_end_lens[b] - seq_len + j.
    accepted [B, A], accepted_lens, kv_cache_end_lens [B] int32; end_lens_out [B] int32 or None:
    the ends behind the accepted rows, may be kv_cache_end_lens itself."""
    _check("kv_accept_drafts", _native().accept(kv_cache, kv_cache_end_lens, seq_len, accepted, accepted_lens,
                                                end_lens_out, stream))


def paged_kv_accept_drafts(kv_cache: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                           seq_len: int, accepted: torch.Tensor, accepted_lens: torch.Tensor,
                           kv_lens_out: Optional[torch.Tensor] = None,
                           kv_scales: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> None:
    """kv_accept_drafts in a paged cache [2, P, TPP, Hkv, D] (float16, or float8_e4m3fn or
    int8 with kv_scales [2, P, Hkv, TPP] float32), by positions through page_table
    [B, 2, M] int32."""
    _check("paged_kv_accept_drafts", _native().paged_accept(kv_cache, page_table, kv_lens, seq_len, accepted,
                                                            accepted_lens, kv_lens_out, kv_scales, stream))


def paged_kv_copy_pages(kv_cache: torch.Tensor, src_pages: torch.Tensor, dst_pages: torch.Tensor,
                        kv_scales: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> None:
    """Page dst_pages[i] of both planes of the pool becomes a copy of page src_pages[i] ([N]
    int32 in [0, P); other entries are skipped), scales too."""
    _check("paged_kv_copy_pages", _native().copy_pages(kv_cache, src_pages, dst_pages, kv_scales, stream))


def paged_kv_fork(kv_cache: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                  ref_counts: torch.Tensor, parents: torch.Tensor, children: torch.Tensor,
                  kv_scales: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Sequence children[i], empty before, becomes a copy of sequence parents[i] ([N] int32):
    whole pages are shared (ref_counts [P] int32 grows), a partly filled last page is copied to
    the lowest free page (one with ref_counts 0). page_table [B, 2, M] int32 and kv_lens [B]
    int32 get the children's rows; pages that an empty child's row still names are given up. A fork
    into a sequence that is not empty, or is itself a parent in this call, is skipped. workspace:
    a uint8 tensor of paged_kv_fork_workspace_size bytes, or None."""
    _check("paged_kv_fork", _native().fork(kv_cache, page_table, kv_lens, ref_counts, parents, children, kv_scales,
                                           workspace, stream))


def paged_kv_fork_workspace_size(num_forks: int, batch: int) -> int:
    """Bytes of workspace that paged_kv_fork needs."""
    lib = _serving.load_serving_library()
    return _check("paged_kv_fork_workspace_size", lib.paged_kv_fork_workspace_size(num_forks, batch))


def paged_kv_free(page_table: torch.Tensor, kv_lens: torch.Tensor, ref_counts: torch.Tensor,
                  sequences: torch.Tensor, tokens_per_page: Optional[int] = None,
                  keep_lens: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Gives up the pages of ``sequences`` ([N] int32): their entries become -1, ref_counts
    shrinks, kv_lens becomes 0. With keep_lens [N] int32 the pages of the first keep_lens[i]
    tokens stay (tokens_per_page is then needed) and kv_lens is cut to that."""
    if tokens_per_page is None:
        if keep_lens is not None:
            raise ValueError("tokens_per_page is needed with keep_lens")
        tokens_per_page = 1        # of no consequence: every page goes
    _check("paged_kv_free", _native().release(page_table, kv_lens, ref_counts, sequences, tokens_per_page, keep_lens,
                                              stream))
