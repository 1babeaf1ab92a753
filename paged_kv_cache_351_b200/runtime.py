"""A paged KV cache on one GPU: the host allocator plus the device pools,
driven through the library's entry points.

This is bookkeeping around libpa: the allocator decides slots and
copy-on-write pairs on the host; the pairs are copied with pa_copy_blocks
and the tokens written with pa_reshape_and_cache (in that order, on one
stream); decode reads through int32 block tables.  Device memory comes from
torch; every byte is moved by the library's kernels.
"""

from __future__ import annotations

from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from . import (PA_DECODE_WS_HEADER_BYTES, Allocator, pa_copy_blocks, pa_decode, pa_decode_cascade,
               pa_decode_cascade_workspace_bytes, pa_decode_fp8, pa_decode_scored, pa_decode_scored_workspace_bytes,
               pa_decode_workspace_bytes, pa_evict, pa_reshape_and_cache, pa_reshape_and_cache_fp8,
               pa_tree_attention, pa_tree_attention_workspace_bytes, pa_tree_commit,
               prepare_decode, prepare_decode_cascade, prepare_decode_fp8, prepare_reshape_and_cache,
               prepare_reshape_and_cache_fp8)

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def _stream(stream, device) -> Optional[torch.cuda.Stream]:
    """A stream argument (None, a torch stream or a raw handle) as torch's."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


class PagedKVCacheGPU:
    """K/V pools [num_blocks, num_kv_heads, block_size, head_size] on one device."""

    def __init__(self, num_blocks: int, num_kv_heads: int, head_size: int, dtype: str = "bf16",
                 block_size: int = 16, free_order: Optional[Sequence[int]] = None, device="cuda",
                 k_scale=None, v_scale=None):
        """dtype "fp8" stores e4m3 codes and needs per-kv-head k_scale/v_scale
        (float32 [num_kv_heads])."""
        self.num_blocks, self.num_kv_heads, self.head_size = num_blocks, num_kv_heads, head_size
        self.block_size, self.dtype, self.device = block_size, dtype, torch.device(device)
        shape = (num_blocks, num_kv_heads, block_size, head_size)
        self.k_cache = torch.empty(shape, dtype=_DT[dtype], device=self.device)
        self.v_cache = torch.empty(shape, dtype=_DT[dtype], device=self.device)
        self.alloc = Allocator(num_blocks, block_size, free_order)
        self._scratch = {}  # (call, stream) -> workspace
        self.k_scale = self.v_scale = None
        if dtype == "fp8":
            if k_scale is None or v_scale is None:
                raise ValueError("an fp8 cache needs k_scale and v_scale")
            self.k_scale = torch.as_tensor(k_scale, dtype=torch.float32).to(self.device).contiguous()
            self.v_scale = torch.as_tensor(v_scale, dtype=torch.float32).to(self.device).contiguous()

    # -- host bookkeeping ------------------------------------------------------
    def add(self, seq: int) -> None:
        self.alloc.add(seq)

    def fork(self, parent: int, child: int) -> None:
        self.alloc.fork(parent, child)

    def free(self, seq: int) -> None:
        self.alloc.free(seq)

    def truncate(self, seq: int, new_len: int) -> None:
        """Give back the slots of a sequence's rejected drafted tokens."""
        self.alloc.truncate(seq, new_len)

    def append(self, seqs: Sequence[int], counts: Sequence[int]) -> Tuple[np.ndarray, np.ndarray]:
        """Reserve slots for counts[k] new tokens of seqs[k]; returns (slots
        int64 [sum(counts)], copy-on-write pairs int64 [n, 2])."""
        return self.alloc.append_batch(seqs, counts)

    def block_tables(self, seqs: Sequence[int], max_blocks: int) -> Tuple[np.ndarray, np.ndarray]:
        return self.alloc.block_tables(seqs, max_blocks)

    # -- device steps -------------------------------------------------------------
    def write(self, slots: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
              pairs: Optional[torch.Tensor] = None, stream=None) -> None:
        """Copy-on-write copies first (they must precede writes into the
        copied blocks), then the tokens' K/V at their slots."""
        if pairs is not None and pairs.shape[0]:
            pa_copy_blocks(self.k_cache, self.v_cache, pairs, stream=stream)
        if self.dtype == "fp8":
            pa_reshape_and_cache_fp8(key, value, self.k_cache, self.v_cache, slots, self.k_scale, self.v_scale,
                                     stream=stream)
        else:
            pa_reshape_and_cache(key, value, self.k_cache, self.v_cache, slots, stream=stream)

    def _workspace(self, call: str, nbytes: int, stream) -> Optional[torch.Tensor]:
        """The zero-filled workspace of one kind of call on ``stream`` (the
        current one if None), grown on demand.  Each stream has its own: it is
        zeroed on the stream that uses it, calls on two streams may overlap,
        and one that is outgrown goes back to its own stream's memory.  A call
        that is captured into a graph gets one of the graph's own memory, whose
        counters the graph zeroes at each replay: graphs share none with each
        other or with calls outside, and none is freed under a graph."""
        if nbytes == 0:
            return None
        dev = self.k_cache.device
        with torch.cuda.device(dev), torch.cuda.stream(_stream(stream, dev)):
            if torch.cuda.is_current_stream_capturing():
                ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
                ws[:PA_DECODE_WS_HEADER_BYTES].zero_()  # (the rest is written before it is used)
                return ws
            key = (call, torch.cuda.current_stream(dev).cuda_stream)
            ws = self._scratch.get(key)
            if ws is None or ws.numel() < nbytes:
                ws = self._scratch[key] = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        return ws

    def workspace(self, num_seqs: int, num_heads: int, max_blocks: int, partition_tokens: int = 0, stream=None):
        """Split scratch for ``decode`` on ``stream`` (the current one if
        None), grown on demand and reused by every such call (zero-filled when
        allocated: its merge counters must start at zero, and every call
        leaves them zero): decodes that may overlap on the GPU must not share
        one."""
        n = pa_decode_workspace_bytes(num_seqs, num_heads, self.num_kv_heads, self.head_size, max_blocks,
                                      partition_tokens)
        return self._workspace("decode", n, stream)

    def prefix_groups(self, seqs: Sequence[int], num_heads: int):
        """Groups of consecutive batch sequences that share leading blocks
        (forks of one prompt), for ``decode_shared``: returns
        (group_start, group_blocks) as int32 numpy arrays and the group width
        to pass as max_group_size (the widest group found, rounded up to a
        power of two, at most 8 query rows per kv head in all)."""
        g = num_heads // self.num_kv_heads
        widest = max(1, 8 // g)
        gs, gb = self.alloc.prefix_groups(seqs, widest)
        sizes = gs[1:] - gs[:-1]
        need = int(sizes[gb > 0].max()) if (gb > 0).any() else 1
        m = 1
        while m < need:
            m *= 2
        if m != widest:
            gs, gb = self.alloc.prefix_groups(seqs, m)
        return gs, gb, m

    def shared_workspace(self, num_seqs: int, num_heads: int, max_group_size: int, partition_tokens: int = 0,
                         stream=None):
        """Zero-filled workspace for ``decode_shared`` on ``stream`` (the
        current one if None), grown on demand and reused by every such call."""
        n = pa_decode_cascade_workspace_bytes(num_seqs, num_heads, self.num_kv_heads, self.head_size, max_group_size,
                                              partition_tokens)
        return self._workspace("decode_shared", n, stream)

    def decode_shared(self, out: torch.Tensor, query: torch.Tensor, block_tables: torch.Tensor,
                      context_lens: torch.Tensor, group_start: torch.Tensor, group_blocks: torch.Tensor,
                      max_group_size: int, scale: float, partition_tokens: int = 0, stream=None,
                      workspace=None) -> torch.Tensor:
        """Decode with each group's shared prompt blocks read once for all
        of its samples (pa_decode_cascade)."""
        if workspace is None:
            workspace = self.shared_workspace(query.shape[0], query.shape[1], max_group_size, partition_tokens, stream)
        pa_decode_cascade(out, query, self.k_cache, self.v_cache, block_tables, context_lens, group_start,
                          group_blocks, max_group_size, scale, self.num_kv_heads, workspace,
                          partition_tokens=partition_tokens, stream=stream)
        return out

    def decode(self, out: torch.Tensor, query: torch.Tensor, block_tables: torch.Tensor,
               context_lens: torch.Tensor, scale: float, partition_tokens: int = 0, stream=None,
               workspace=None) -> torch.Tensor:
        if workspace is None:
            workspace = self.workspace(query.shape[0], query.shape[1], block_tables.shape[1], partition_tokens, stream)
        if self.dtype == "fp8":
            pa_decode_fp8(out, query, self.k_cache, self.v_cache, block_tables, context_lens, scale,
                          self.num_kv_heads, self.k_scale, self.v_scale, workspace=workspace,
                          partition_tokens=partition_tokens, stream=stream)
        else:
            pa_decode(out, query, self.k_cache, self.v_cache, block_tables, context_lens, scale, self.num_kv_heads,
                      workspace=workspace, partition_tokens=partition_tokens, stream=stream)
        return out

    # -- speculative decoding ---------------------------------------------------------
    def tree_attention(self, out: torch.Tensor, query: torch.Tensor, block_tables: torch.Tensor,
                       context_lens: torch.Tensor, query_start: torch.Tensor, tree_mask: torch.Tensor,
                       max_query_len: int, scale: float, stream=None, workspace=None) -> torch.Tensor:
        """Attention of every sequence's drafted tokens over its cache
        (pa_tree_attention; the drafted tokens are already written).  Without
        a ``workspace``, one kept here for the stream is used."""
        if workspace is None:
            n = pa_tree_attention_workspace_bytes(query.shape[1], self.num_kv_heads, self.head_size, max_query_len)
            workspace = self._workspace("tree_attention", n, stream)
        pa_tree_attention(out, query, self.k_cache, self.v_cache, block_tables, context_lens, query_start, tree_mask,
                          max_query_len, scale, self.num_kv_heads, workspace=workspace, stream=stream)
        return out

    def tree_commit(self, block_tables: torch.Tensor, context_lens: torch.Tensor, query_start: torch.Tensor,
                    accepted: torch.Tensor, num_accepted: torch.Tensor, stream=None) -> None:
        """Move the accepted drafted tokens' K/V behind the context
        (pa_tree_commit); ``truncate`` then drops the rest of the draft."""
        pa_tree_commit(self.k_cache, self.v_cache, block_tables, context_lens, query_start, accepted, num_accepted,
                       stream=stream)

    # -- bounded caches -----------------------------------------------------------------
    def decode_scored(self, out: torch.Tensor, scores: torch.Tensor, query: torch.Tensor,
                      block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                      partition_tokens: int = 0, stream=None, workspace=None) -> torch.Tensor:
        """decode, with every cached token's attention weight added to
        ``scores`` [B, num_kv_heads, S] (pa_decode_scored).  Without a
        ``workspace``, one kept here for the stream is used."""
        if workspace is None:
            n = pa_decode_scored_workspace_bytes(query.shape[0], query.shape[1], self.num_kv_heads, self.head_size,
                                                 block_tables.shape[1], partition_tokens)
            workspace = self._workspace("decode_scored", n, stream)
        pa_decode_scored(out, scores, query, self.k_cache, self.v_cache, block_tables, context_lens, scale,
                         self.num_kv_heads, workspace, k_scale=self.k_scale, v_scale=self.v_scale,
                         partition_tokens=partition_tokens, stream=stream)
        return out

    def evict(self, seqs: Sequence[int], keep: Sequence[int], scores: torch.Tensor, scores_out: torch.Tensor,
              num_sink: int = 0, num_recent: int = 0, stream=None) -> torch.Tensor:
        """Shorten sequences to ``keep[k]`` tokens each by accumulated weight
        (row k of ``scores``; pa_evict): the allocator gives them fresh
        blocks, the kept tokens move there, and ``scores_out`` gets their
        scores.  Returns the kept positions, int32 [n, num_kv_heads, *].
        Raises OutOfBlocksError, with nothing changed, when the fresh blocks
        do not all fit beside the old ones."""
        lens = [self.alloc.length(s) for s in seqs]
        new = [min(int(k), n) for k, n in zip(keep, lens)]
        if len(keep) != len(seqs) or min(new, default=0) < 0 or num_sink < 0 or num_recent < 0:
            raise ValueError("one length >= 0 per sequence, num_sink and num_recent >= 0")
        # everything pa_evict would refuse, before the allocator changes
        if len(new) > 65535:
            raise ValueError("at most 65535 sequences in one call")
        for t, need, what in ((scores, max(lens, default=0), "scores"), (scores_out, max(new, default=0), "scores_out")):
            if (tuple(t.shape[:2]) != (len(new), self.num_kv_heads) or t.dim() != 3 or t.shape[2] < need or
                    t.dtype != torch.float32 or t.device != self.k_cache.device or t.stride(2) != 1 or
                    t.stride(1) < t.shape[2] or t.stride(0) < t.shape[2]):
                raise ValueError(f"{what} must be float32 [{len(new)}, {self.num_kv_heads}, at least {need}] on "
                                 f"{self.k_cache.device} with contiguous rows")
        if scores.numel() and scores.data_ptr() == scores_out.data_ptr():
            raise ValueError("scores_out must not be scores")
        bs = self.block_size
        src, ctx = self.alloc.block_tables(seqs, max([(n + bs - 1) // bs for n in lens] + [1]))
        width = max([(n + bs - 1) // bs for n in new] + [1])
        stream = _stream(stream, self.k_cache.device)
        # the uploads belong to the stream that reads them; all device memory
        # is taken before the allocator changes
        with torch.cuda.stream(stream):
            kept = torch.empty(len(new), self.num_kv_heads, max(new, default=0), dtype=torch.int32, device=self.device)
            up = [torch.from_numpy(x).to(self.device) for x in (src, ctx, np.asarray(new, np.int32))]
            dst = torch.empty(len(new), width, dtype=torch.int32, device=self.device)
            dst.copy_(torch.from_numpy(self.alloc.compact(seqs, new, width)))
            pa_evict(self.k_cache, self.v_cache, up[0], up[1], scores, dst, up[2], num_sink, num_recent, scores_out,
                     kept, stream=stream)
        return kept

    def prepare_step(self, slots: torch.Tensor, key: torch.Tensor, value: torch.Tensor, out: torch.Tensor,
                     query: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                     partition_tokens: int = 0, stream=None, workspace=None, groups=None):
        """One serving step (the new tokens' cache write, then the decode)
        over fixed buffers, as prepared calls (descriptors built once): the
        returned function runs the step again on the buffers' current
        contents.  ``groups``: (group_start, group_blocks, max_group_size)
        device tensors and width for a shared-prefix decode."""
        if self.dtype == "fp8":
            write = prepare_reshape_and_cache_fp8(key, value, self.k_cache, self.v_cache, slots, self.k_scale,
                                                  self.v_scale, stream=stream)
        else:
            write = prepare_reshape_and_cache(key, value, self.k_cache, self.v_cache, slots, stream=stream)
        if groups is not None:
            gs, gb, mg = groups
            if workspace is None:
                workspace = self.shared_workspace(query.shape[0], query.shape[1], mg, partition_tokens, stream)
            dec = prepare_decode_cascade(out, query, self.k_cache, self.v_cache, block_tables, context_lens, gs, gb,
                                         mg, scale, self.num_kv_heads, workspace, partition_tokens, stream=stream)
        else:
            if workspace is None:
                workspace = self.workspace(query.shape[0], query.shape[1], block_tables.shape[1], partition_tokens,
                                           stream)
            if self.dtype == "fp8":
                dec = prepare_decode_fp8(out, query, self.k_cache, self.v_cache, block_tables, context_lens, scale,
                                         self.num_kv_heads, self.k_scale, self.v_scale, workspace, partition_tokens,
                                         stream=stream)
            else:
                dec = prepare_decode(out, query, self.k_cache, self.v_cache, block_tables, context_lens, scale,
                                     self.num_kv_heads, workspace, partition_tokens, stream=stream)
        return PreparedStep(write if slots.numel() > 0 else None, dec)


class PreparedStep:
    """A serving step as prepared library calls: ``write`` (the new tokens'
    cache write, None when the step appends nothing) and ``decode``; calling
    the step runs both, in that order, on the stream they were prepared
    with."""

    def __init__(self, write, decode):
        self.write = write
        self.decode = decode

    def __call__(self) -> None:
        if self.write is not None:
            self.write()
        self.decode()
