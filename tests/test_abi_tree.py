"""Argument checks of the speculative-decoding calls: each refusal is an error
before anything is launched (no GPU needed)."""

import pytest
import torch

import paged_kv_cache_351_b200 as pa

INVALID, UNSUPPORTED = 1, 2


def _tree(B=2, T=5, H=4, hk=2, D=128, nb=6, dtype=torch.bfloat16, max_q=3, words=1):
    return dict(out=torch.empty(T, H, D, dtype=dtype), query=torch.empty(T, H, D, dtype=dtype),
                k_cache=torch.empty(nb, hk, 16, D, dtype=dtype), v_cache=torch.empty(nb, hk, 16, D, dtype=dtype),
                block_tables=torch.zeros(B, 4, dtype=torch.int32), context_lens=torch.zeros(B, dtype=torch.int32),
                query_start=torch.zeros(B + 1, dtype=torch.int32),
                tree_mask=torch.zeros(T, words, dtype=torch.int32), max_query_len=max_q, scale=0.1, num_kv_heads=hk)


BAD = [
    (INVALID, dict(num_kv_heads=3)),
    (INVALID, dict(query=torch.empty(5, 3, 128, dtype=torch.bfloat16))),
    (INVALID, dict(query=torch.empty(5, 4, 128))),
    (INVALID, dict(query=torch.empty(5, 4, 132, dtype=torch.bfloat16)[:, :, 2:130])),
    (INVALID, dict(out=torch.empty(4, 4, 128, dtype=torch.bfloat16))),
    (INVALID, dict(context_lens=torch.zeros(2, dtype=torch.int64))),
    (INVALID, dict(context_lens=torch.zeros(4, dtype=torch.int32)[::2])),
    (INVALID, dict(query_start=torch.zeros(2, dtype=torch.int32))),
    (INVALID, dict(block_tables=torch.zeros(3, 4, dtype=torch.int32))),
    (INVALID, dict(block_tables=torch.zeros(4, 2, dtype=torch.int32).t())),
    (INVALID, dict(tree_mask=torch.zeros(5, 1, dtype=torch.int64))),
    (INVALID, dict(tree_mask=torch.zeros(4, 1, dtype=torch.int32))),
    (INVALID, dict(tree_mask=torch.zeros(5, 0, dtype=torch.int32))),
    (INVALID, dict(max_query_len=6)),
    (INVALID, dict(max_query_len=0)),
    (INVALID, dict(max_query_len=-1)),
    (INVALID, dict(scale=0.0)),
    (INVALID, dict(scale=float("nan"))),
    (INVALID, dict(scale=float("inf"))),
    (INVALID, dict(partition_tokens=-2)),
    (UNSUPPORTED, dict(partition_tokens=512)),
    (INVALID, dict(v_cache=torch.empty(5, 2, 16, 128, dtype=torch.bfloat16))),
    (UNSUPPORTED, dict(k_cache=torch.empty(6, 2, 32, 128, dtype=torch.bfloat16),
                       v_cache=torch.empty(6, 2, 32, 128, dtype=torch.bfloat16))),
]


@pytest.mark.parametrize("status,change", BAD)
def test_tree_attention_refuses(status, change):
    args = _tree()
    part = change.get("partition_tokens", 0)
    args.update({k: v for k, v in change.items() if k != "partition_tokens"})
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.pa_tree_attention(**args, partition_tokens=part, stream=0)
    assert e.value.status == status


def test_tree_attention_refuses_what_it_has_no_kernel_for():
    for change, args in (("group of 3", _tree(H=6)), ("fp8", _tree(dtype=torch.float8_e4m3fn)),
                         ("long draft", _tree(T=1025, max_q=1025, words=33))):
        if change == "fp8":
            args["query"] = args["out"] = torch.empty(5, 4, 128, dtype=torch.bfloat16)
        with pytest.raises(pa.PagedAttentionError) as e:
            pa.pa_tree_attention(**args, stream=0)
        assert e.value.status == UNSUPPORTED, change


def test_tree_attention_with_nothing_to_do():
    pa.pa_tree_attention(**_tree(T=0, max_q=0, words=0), stream=0)
    pa.pa_tree_attention(**_tree(B=0), stream=0)


def test_tree_attention_refuses_a_misaligned_workspace():
    args = _tree()
    ws = torch.zeros(1 << 17, dtype=torch.uint8)
    ws = ws[(16 - ws.data_ptr()) % 256:][:1 << 16]
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.pa_tree_attention(**args, workspace=ws, stream=0)
    assert e.value.status == INVALID


def test_workspace_size_arguments():
    for bad in ((0, 1, 128, 4), (4, 0, 128, 4), (4, 3, 128, 4), (4, 2, 0, 4), (4, 2, 128, -1)):
        with pytest.raises(pa.PagedAttentionError) as e:
            pa.pa_tree_attention_workspace_bytes(*bad)
        assert e.value.status == INVALID


def _commit(B=2, hk=2, D=128, nb=6, P=3, dtype=torch.bfloat16):
    return dict(k_cache=torch.empty(nb, hk, 16, D, dtype=dtype), v_cache=torch.empty(nb, hk, 16, D, dtype=dtype),
                block_tables=torch.zeros(B, 4, dtype=torch.int32), context_lens=torch.zeros(B, dtype=torch.int32),
                query_start=torch.zeros(B + 1, dtype=torch.int32), accepted=torch.zeros(B, P, dtype=torch.int32),
                num_accepted=torch.zeros(B, dtype=torch.int32))


@pytest.mark.parametrize("change", [
    dict(v_cache=torch.empty(6, 2, 16, 128)),
    dict(context_lens=torch.zeros(3, dtype=torch.int32)),
    dict(query_start=torch.zeros(2, dtype=torch.int32)),
    dict(accepted=torch.zeros(3, 3, dtype=torch.int32)),
    dict(accepted=torch.zeros(2, 3, dtype=torch.int64)),
    dict(accepted=torch.zeros(3, 2, dtype=torch.int32).t()),
    dict(num_accepted=torch.zeros(2, 1, dtype=torch.int32)),
    dict(block_tables=torch.zeros(2, 4, dtype=torch.int64)),
])
def test_commit_refuses(change):
    args = _commit()
    args.update(change)
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.pa_tree_commit(**args, stream=0)
    assert e.value.status == INVALID


def test_commit_with_nothing_to_do():
    pa.pa_tree_commit(**_commit(B=0), stream=0)


def test_more_kv_heads_than_a_grid_has():
    for fn, args in ((pa.pa_tree_attention, _tree(T=1, H=65536, hk=65536, D=64, nb=1, max_q=1)),
                     (pa.pa_tree_commit, _commit(hk=65536, D=64, nb=1))):
        with pytest.raises(pa.PagedAttentionError) as e:
            fn(**args, stream=0)
        assert e.value.status == UNSUPPORTED


def test_tables_too_long_for_32_bit_positions():
    """(untouched memory, so only addresses are taken)"""
    long = torch.empty(1, (2**31 - 2**24) // 16, dtype=torch.int32)
    tree, commit = _tree(B=1), _commit(B=1)
    tree["block_tables"] = commit["block_tables"] = long
    for fn, args in ((pa.pa_tree_attention, tree), (pa.pa_tree_commit, commit)):
        with pytest.raises(pa.PagedAttentionError) as e:
            fn(**args, stream=0)
        assert e.value.status == UNSUPPORTED
