"""Argument checks of the scored decode and of eviction: each refusal is an
error before anything is launched (no GPU needed)."""

import pytest
import torch

import paged_kv_cache_351_b200 as pa

INVALID, UNSUPPORTED = 1, 2


def _scored(B=2, H=4, hk=2, D=128, nb=6, dtype=torch.bfloat16, S=64):
    qd = torch.bfloat16 if dtype == torch.float8_e4m3fn else dtype
    ws = torch.zeros((1 << 16) + 256, dtype=torch.uint8)
    ws = ws[(-ws.data_ptr()) % 256:][:1 << 16]
    return dict(out=torch.empty(B, H, D, dtype=qd), scores=torch.zeros(B, hk, S), query=torch.empty(B, H, D, dtype=qd),
                k_cache=torch.empty(nb, hk, 16, D, dtype=dtype), v_cache=torch.empty(nb, hk, 16, D, dtype=dtype),
                block_tables=torch.zeros(B, 4, dtype=torch.int32), context_lens=torch.zeros(B, dtype=torch.int32),
                scale=0.1, num_kv_heads=hk, workspace=ws, stream=0)


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(scores=torch.zeros(2, 4, 64))),
    (INVALID, dict(scores=torch.zeros(3, 2, 64))),
    (INVALID, dict(scores=torch.zeros(2, 2, 64, dtype=torch.bfloat16))),
    (INVALID, dict(scores=torch.zeros(2, 2, 128)[:, :, ::2])),
    (INVALID, dict(scores=torch.zeros(2, 128))),
    (INVALID, dict(scores=torch.zeros(1, 2, 64).expand(2, 2, 64))),
    (INVALID, dict(workspace=None)),
    (UNSUPPORTED, dict(partition_tokens=64)),
    (INVALID, dict(partition_tokens=-3)),
    (INVALID, dict(k_scale=torch.ones(2), v_scale=torch.ones(2))),
    (INVALID, dict(query=torch.empty(2, 4, 64, dtype=torch.bfloat16))),
    (INVALID, dict(scale=float("inf"))),
    (INVALID, dict(num_kv_heads=4)),
])
def test_scored_decode_refuses(status, change):
    args = _scored()
    args.update(change)
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.pa_decode_scored(**args)
    assert e.value.status == status


def test_scored_decode_refuses_an_fp8_cache_without_scales_and_odd_groups():
    for args, status in ((_scored(dtype=torch.float8_e4m3fn), INVALID), (_scored(H=6), UNSUPPORTED)):
        with pytest.raises(pa.PagedAttentionError) as e:
            pa.pa_decode_scored(**args)
        assert e.value.status == status


def test_scored_decode_with_nothing_to_do():
    pa.pa_decode_scored(**_scored(B=0))


def test_scored_workspace_arguments():
    for bad, status in (((2, 4, 3, 128, 4), INVALID), ((-1, 4, 2, 128, 4), INVALID), ((2, 4, 2, 128, -1), INVALID),
                        ((2, 4, 2, 128, 4, 16), UNSUPPORTED), ((2, 4, 2, 128, 4, -2), INVALID)):
        with pytest.raises(pa.PagedAttentionError) as e:
            pa.pa_decode_scored_workspace_bytes(*bad)
        assert e.value.status == status


def _evict(B=2, hk=2, D=128, nb=6, dtype=torch.bfloat16):
    return dict(k_cache=torch.empty(nb, hk, 16, D, dtype=dtype), v_cache=torch.empty(nb, hk, 16, D, dtype=dtype),
                block_tables=torch.zeros(B, 4, dtype=torch.int32), context_lens=torch.zeros(B, dtype=torch.int32),
                scores=torch.zeros(B, hk, 64), dst_tables=torch.zeros(B, 2, dtype=torch.int32),
                keep_lens=torch.zeros(B, dtype=torch.int32), num_sink=1, num_recent=2,
                scores_out=torch.zeros(B, hk, 64), kept_out=torch.zeros(B, hk, 32, dtype=torch.int32), stream=0)


@pytest.mark.parametrize("change", [
    dict(v_cache=torch.empty(6, 2, 16, 128)),
    dict(context_lens=torch.zeros(3, dtype=torch.int32)),
    dict(keep_lens=torch.zeros(2, dtype=torch.int64)),
    dict(keep_lens=torch.zeros(1, dtype=torch.int32)),
    dict(dst_tables=torch.zeros(3, 2, dtype=torch.int32)),
    dict(block_tables=torch.zeros(4, 2, dtype=torch.int32).t()),
    dict(scores=torch.zeros(2, 1, 64)),
    dict(scores=torch.zeros(2, 2, 64, dtype=torch.float64).float().double()[:, :, :1].int().expand(2, 2, 64)),
    dict(scores_out=torch.zeros(2, 2, 128)[:, :, ::2]),
    dict(kept_out=torch.zeros(2, 2, 32)),
    dict(num_sink=-1),
    dict(num_recent=-1),
])
def test_evict_refuses(change):
    args = _evict()
    args.update(change)
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.pa_evict(**args)
    assert e.value.status == INVALID


def test_evict_refuses_to_compact_scores_in_place():
    args = _evict()
    args["scores_out"] = args["scores"]
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.pa_evict(**args)
    assert e.value.status == INVALID


def test_evict_with_nothing_to_do():
    pa.pa_evict(**_evict(B=0))


def test_evict_refuses_more_kv_heads_than_a_grid_has():
    args = _evict(B=1, hk=65536, D=64, nb=1)
    args.update(scores=torch.zeros(1, 65536, 1), scores_out=torch.ones(1, 65536, 1),
                kept_out=torch.zeros(1, 65536, 1, dtype=torch.int32))
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.pa_evict(**args)
    assert e.value.status == UNSUPPORTED


def test_tables_too_long_for_32_bit_positions():
    """(untouched memory, so only addresses are taken)"""
    long = torch.empty(1, (2**31 - 2**24) // 16, dtype=torch.int32)
    scored = _scored(B=1)
    scored.update(block_tables=long)
    src, dst = _evict(B=1), _evict(B=1)
    src["block_tables"], dst["dst_tables"] = long, long
    for fn, args in ((pa.pa_decode_scored, scored), (pa.pa_evict, src), (pa.pa_evict, dst)):
        with pytest.raises(pa.PagedAttentionError) as e:
            fn(**args)
        assert e.value.status == UNSUPPORTED
