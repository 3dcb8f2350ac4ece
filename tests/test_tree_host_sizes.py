"""The binding's record of workspace sizes, which goes by the device, without one."""
import pytest
import torch

import block_sparse_attention_idx_b200 as msa


def test_a_size_is_recorded_for_the_device_that_it_was_computed_on(monkeypatch):
    """Tensors on another device than the current one are refused before a size of the current one is recorded for
    theirs: the right call that follows gets its own device's size."""
    here = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: here[0])
    monkeypatch.setattr(msa, "msa_tree_workspace_size", lambda op, dims, T: (148 if here[0] == 0 else 160) * 1000)
    msa._tree_ws_size.cache_clear()
    size = lambda dev: msa._tree_ws_size(msa.MSA_OP_TREE_ATTN, 1, 100, 4, 2, 64, 32, 32, 4, 3, dev)  # noqa: E731
    try:
        assert size(0) == 148000
        with pytest.raises(ValueError, match="current CUDA device is cuda:0"):
            size(1)
        here[0] = 1
        assert size(1) == 160000
    finally:
        msa._tree_ws_size.cache_clear()
