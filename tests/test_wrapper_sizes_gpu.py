"""Tensor sizes past 32 bits: refused by the entry points before anything is launched."""
import pytest
import torch

import sparse_mla_attention_fwd_gb300 as smla
from test_paged_ops_gpu import i32

pytestmark = pytest.mark.gpu

WIDE = 2 ** 32 + 64


def test_tables_and_layers_past_32_bits():
    none, table = i32([]), torch.empty((0, WIDE), dtype=torch.int32, device="cuda")
    pool, q = (torch.zeros((64, n, 576), dtype=torch.bfloat16, device="cuda") for n in (1, 2))
    cu, keep = i32([0]), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    for call in (lambda: smla.sparse_mla_plan_pages(none, none, table, i32([0, 1]), 4),
                 lambda: smla.sparse_mla_chunk_fwd_paged(q, pool, table, cu, none),
                 lambda: smla.sparse_mla_tree_fwd_paged(q, pool, table, cu, none, torch.zeros((64, 1), dtype=torch.int32, device="cuda")),
                 lambda: smla.sparse_mla_commit_tree(keep, none, cu, none, table, pool)):
        with pytest.raises(ValueError, match="max_blocks.* 32 bits"):
            call()
    layers = torch.zeros((1, 64, 1, 576), dtype=torch.bfloat16, device="cuda").expand(2 ** 32 + 1, -1, -1, -1)
    with pytest.raises(ValueError, match="layers.* 32 bits"):
        smla.sparse_mla_commit_tree(i32([[0, 2]]), i32([2]), i32([0, 3]), i32([9]), i32([[0, 1]]), layers)
