"""Eviction through PagedKVCacheGPU: what the call refuses, it refuses before
the allocator changes; counts past 32 bits mean "all"."""

import pytest
import torch

import paged_kv_cache_351_b200 as pa
from paged_kv_cache_351_b200.runtime import PagedKVCacheGPU


def test_more_sequences_than_a_launch_has_change_nothing():
    """(a host cache, whose memory is never touched: only the bookkeeping counts)"""
    n = 65536
    kv = PagedKVCacheGPU(2 * n, 1, 64, "bf16", device="cpu")
    seqs = list(range(n))
    for s in seqs:
        kv.add(s)
    kv.append(seqs, [1] * n)
    tables = [kv.alloc.block_table(s) for s in (0, 1, n - 1)]
    scores = torch.zeros(n, 1, 1)
    with pytest.raises(ValueError):
        kv.evict(seqs, [1] * n, scores, torch.ones(n, 1, 1))
    assert [kv.alloc.block_table(s) for s in (0, 1, n - 1)] == tables and kv.alloc.num_free() == n


@pytest.mark.parametrize("many", [2**31, 2**32, 2**32 + 1, 2**63 - 1])
def test_counts_past_32_bits_are_not_taken_modulo(many):
    assert pa._count(many) == 2**31 - 1 and pa._count(-many) < 0


@pytest.mark.gpu
@pytest.mark.parametrize("sink,recent,kept", [(0, 2**40, list(range(90, 100))), (2**32 + 1, 3, [0, 1, 2, 3, 4, 5, 6, 97, 98, 99]),
                                              (2**63 - 1, 2**63 - 1, list(range(90, 100)))])
def test_all_recent_or_all_first(sink, recent, kept):
    kv = PagedKVCacheGPU(16, 2, 64, "f32")
    kv.add(0)
    kv.append([0], [100])
    s = torch.zeros(1, 2, 128, device="cuda")
    s[:, :, 50] = 1.0
    got = kv.evict([0], [10], s, torch.ones_like(s), num_sink=sink, num_recent=recent)
    assert got.tolist() == [[kept, kept]] and kv.alloc.length(0) == 10
