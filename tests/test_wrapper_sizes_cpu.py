"""The Python entry points refuse sizes that do not fit the C interface's 32-bit integers, into which ctypes would wrap them."""
import pytest
import torch

import sparse_mla_attention_fwd_gb300 as smla
from sparse_mla_attention_fwd_gb300.native_build import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return smla.load_library()


I = torch.zeros(4, dtype=torch.int32)
TABLE = torch.zeros((4, 2), dtype=torch.int32)
B = torch.zeros((4, 1, 576), dtype=torch.bfloat16)

CALLS = {
    "sparse_mla_fwd": ((B, B, TABLE), ("d_v",)),
    "sparse_mla_fwd_paged": ((B, B, TABLE, TABLE), ("page_block", "s_q_per_req", "d_v")),
    "sparse_mla_fwd_paged_splitkv_static": ((B, B, TABLE, TABLE, 2), ("page_block", "s_q_per_req", "d_v")),
    "sparse_mla_bwd": ((B, B, B, B, TABLE, I.float()), ("d_v",)),
    "sparse_mla_plan_pages": ((I, I, TABLE, I, 4), ("page_block",)),
    "sparse_mla_chunk_fwd_paged": ((B, B, TABLE, I, I), ("page_block", "d_v")),
    "sparse_mla_tree_fwd_paged": ((B, B, TABLE, I, I, I.view(4, 1)), ("page_block", "d_v")),
    "sparse_mla_commit_tree": ((TABLE, I, I, I, TABLE, B), ("page_block",)),
}


@pytest.mark.parametrize("value", [2 ** 32 + 64, 2 ** 32 + 512, 2 ** 31, -2 ** 32 + 64])
@pytest.mark.parametrize("call,name", [(call, name) for call, (_, names) in CALLS.items() for name in names])
def test_sizes_past_32_bits(call, name, value):
    with pytest.raises(ValueError, match=name + ".* 32 bits"):
        getattr(smla, call)(*CALLS[call][0], **{name: value})


def test_splits_past_32_bits():
    with pytest.raises(ValueError, match="n_split.* 32 bits"):
        smla.sparse_mla_fwd_paged_splitkv_static(B, B, TABLE, TABLE, 2 ** 32 + 2)
    with pytest.raises(ValueError, match="n_chunks.* 32 bits"):
        smla.sparse_mla_fwd_host(B, B, TABLE, device="cuda:0", n_chunks=2 ** 32 + 8)


def test_sizes_that_fit_come_to_the_other_checks():
    for call, (args, names) in CALLS.items():
        for name in names:
            with pytest.raises(ValueError) as e:
                getattr(smla, call)(*args, **{name: 64})
            assert "32 bits" not in str(e.value)
