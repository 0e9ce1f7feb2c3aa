"""B200-native (sm_100a) paged decode attention: the cache write and the
decode-step attention over a block-table-addressed KV cache.

The compute lives in ``libpa.so`` (CUDA kernels behind the C ABI of
``include/pa.h``); this package only marshals torch tensors into those calls.

    from paged_kv_cache_444_b200 import pa_reshape_and_cache, pa_decode
"""
from __future__ import annotations

import contextlib

import torch

from ._lib import (DecodePlan, HostStep, PagedAttentionError, load, pa_check_error, pa_copy_blocks, pa_decode,
                   pa_decode_fp8, pa_decode_noalloc, pa_decode_shared_prefix, pa_decode_split,
                   pa_decode_split_fp8, pa_decode_weights, pa_evict_commit, pa_evict_compact,
                   pa_evict_select,
                   pa_prefill, pa_prompt_attention, pa_prompt_weights, pa_reduce,
                   pa_reshape_and_cache, pa_reshape_and_cache_fp8, pa_selftest_wait_timeout, _stream)

__all__ = [
    "PagedAttentionError", "load", "pa_reshape_and_cache", "pa_decode", "pa_decode_split",
    "pa_reduce", "pa_check_error", "pa_decode_noalloc", "pa_decode_shared_prefix",
    "pa_copy_blocks", "pa_reshape_and_cache_fp8", "pa_decode_fp8", "pa_decode_split_fp8",
    "pa_prefill", "pa_prompt_attention", "pa_prompt_weights", "pa_decode_weights",
    "pa_evict_select", "pa_evict_compact", "pa_evict_commit", "pa_selftest_wait_timeout", "SplitWorkspace", "WeightsWorkspace",
    "EvictionState", "decode_step", "prompt_step", "HostStep", "DecodePlan",
]


class SplitWorkspace:
    """Caller-owned fp32 scratch for pa_decode_split / pa_reduce
    (tmp_out [S, H, P, D], max_logits and exp_sums [S, H, P])."""

    def __init__(self, num_seqs: int, num_heads: int, head_dim: int, max_partitions: int,
                 device: torch.device | str):
        shape = (num_seqs, num_heads, max_partitions)
        self.tmp_out = torch.empty(shape + (head_dim,), dtype=torch.float32, device=device)
        self.max_logits = torch.empty(shape, dtype=torch.float32, device=device)
        self.exp_sums = torch.empty(shape, dtype=torch.float32, device=device)

    @property
    def max_partitions(self) -> int:
        return self.max_logits.shape[-1]


class WeightsWorkspace:
    """Caller-owned scratch for pa_decode_weights (one for calls that follow one
    another; calls that may overlap on the GPU need one each)."""

    def __init__(self, num_seqs: int, num_heads: int, head_dim: int, max_blocks_per_seq: int,
                 device: torch.device | str, block_size: int = 16):
        n = load().pa_decode_weights_workspace_bytes(num_seqs, num_heads, head_dim,
                                                     max_blocks_per_seq, block_size)
        if n < 0:
            raise ValueError("bad workspace sizes")
        self.buffer = torch.empty(max(n, 1), dtype=torch.uint8, device=device)

    @classmethod
    def for_call(cls, query: torch.Tensor, key_cache: torch.Tensor,
                 block_tables: torch.Tensor) -> "WeightsWorkspace":
        """The workspace of a call with these tensors."""
        S, H, D = query.shape
        return cls(S, H, D, block_tables.shape[1], query.device, key_cache.shape[1])


def _pool_of(stream, device):
    """Context whose allocations come from the memory pool of the stream that a
    call is given (None: the current one).  The caching allocator hands memory
    freed on a stream to that stream's next tensor at once, so a buffer from the
    current stream's pool may be in use there while the given stream writes it."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)    # 0 and 1: the default stream
        stream = (torch.cuda.ExternalStream(handle, device) if handle > 1
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


def decode_step(query, key, value, key_cache, value_cache, slot_mapping, block_tables,
                context_lens, scale: float, out: torch.Tensor | None = None,
                partition_size: int = 0, workspace: SplitWorkspace | None = None,
                stream=None) -> torch.Tensor:
    """One decode step of one attention layer: write this step's K/V rows
    (pa_reshape_and_cache), then attend (pa_decode, or pa_decode_split +
    pa_reduce when partition_size > 0).  All tensors live on one CUDA device.
    What is allocated here belongs to `stream`; the returned out may be used on
    the current stream too, once that has waited for `stream`."""
    if out is None:
        with _pool_of(stream, query.device):
            out = torch.empty_like(query)
        if stream is not None:
            out.record_stream(torch.cuda.current_stream(query.device))
    if key is not None and key.shape[0] > 0:
        pa_reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, stream)
    if partition_size > 0:
        if workspace is None:
            bs = key_cache.shape[1]
            P = (block_tables.shape[1] * bs + partition_size - 1) // partition_size
            with _pool_of(stream, query.device):
                workspace = SplitWorkspace(query.shape[0], query.shape[1], query.shape[2], P,
                                           query.device)
        pa_decode_split(workspace.tmp_out, workspace.max_logits, workspace.exp_sums, query,
                        key_cache, value_cache, block_tables, context_lens, scale,
                        partition_size, stream)
        pa_reduce(out, workspace.tmp_out, workspace.max_logits, workspace.exp_sums,
                  context_lens, partition_size, stream)
    else:
        pa_decode(out, query, key_cache, value_cache, block_tables, context_lens, scale, stream)
    return out


def prompt_step(query, key, value, key_cache, value_cache, slot_mapping, seq_starts, scale: float,
                out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                weights: torch.Tensor | None = None, window: int | None = None,
                stream=None) -> torch.Tensor:
    """The first step of packed prompts in one attention layer: write their K/V
    rows into the cache (pa_reshape_and_cache; key_cache None: no write), attend
    (pa_prompt_attention) and, when weights [S, Hk, max_tokens] is given, set the
    attention weight each token receives from the last `window` tokens of its
    prompt, all of them if None (pa_prompt_weights).  All tensors live on one CUDA
    device.  What is allocated here belongs to `stream`; the returned out may be
    used on the current stream too, once that has waited for `stream`."""
    T, H, _ = query.shape
    if out is None:
        with _pool_of(stream, query.device):
            out = torch.empty(query.shape, dtype=query.dtype, device=query.device)
        if stream is not None:
            out.record_stream(torch.cuda.current_stream(query.device))
    if weights is not None and lse is None:
        with _pool_of(stream, query.device):
            lse = torch.empty((T, H), dtype=torch.float32, device=query.device)
    if key_cache is not None:
        pa_reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, stream)
    pa_prompt_attention(out, lse, query, key, value, seq_starts, scale, stream)
    if weights is not None:
        pa_prompt_weights(weights, query, key, lse, seq_starts, scale,
                          max(T, 1) if window is None else window, stream)
    return out


class EvictionState:
    """What one attention layer keeps to hold its sequences to `budget` cached
    tokens: the attention weight each slot's token has received (filled by
    pa_prompt_weights and pa_decode_weights), the tokens' positions, and the
    buffers of pa_evict_select.  The first `sink` tokens of a sequence and its
    latest `recent` ones always stay.  For a new sequence in row s, set
    recorded_lens[s] to 0."""

    def __init__(self, num_seqs: int, num_kv_heads: int, max_tokens: int, budget: int,
                 device: torch.device | str, sink: int = 4, recent: int = 0):
        if min(sink, recent) < 0 or sink + recent > budget:
            raise ValueError("sink + recent must lie within the budget")
        rows = (num_seqs, num_kv_heads)
        i32 = dict(dtype=torch.int32, device=device)
        self.sink, self.recent = int(sink), int(recent)
        self.weights = torch.zeros(rows + (max_tokens,), dtype=torch.float32, device=device)
        self.positions = torch.zeros(rows + (max_tokens,), **i32)
        self.recorded_lens = torch.zeros(num_seqs, **i32)
        self.source = torch.empty(rows + (budget,), **i32)
        self.new_lens = torch.empty(num_seqs, **i32)

    def evict(self, key_cache, value_cache, block_tables, context_lens, seq_lens) -> None:
        """Evict down to the budget on the current stream: select, move the kept
        rows to the front, and set context_lens to the new lengths.  seq_lens [S]
        int32 counts the tokens each sequence has had in all (it must not share
        storage with context_lens).  A length outside [0, max_tokens] is reported
        (pa_check_error) and stays, with all of its sequence.  Capturable in a
        CUDA graph."""
        apart = abs(seq_lens.data_ptr() - context_lens.data_ptr())
        if apart < context_lens.element_size() * context_lens.numel():
            raise ValueError("seq_lens must not share storage with context_lens")
        pa_evict_select(self.source, self.new_lens, self.weights, self.positions, context_lens,
                        self.recorded_lens, seq_lens, self.sink, self.recent)
        pa_evict_compact(key_cache, value_cache, self.weights, self.positions, self.source,
                         self.new_lens, block_tables, context_lens, self.recorded_lens, seq_lens)
        pa_evict_commit(context_lens, self.recorded_lens, self.new_lens)
