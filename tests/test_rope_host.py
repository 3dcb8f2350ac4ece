"""A rotary call whose rows lie further apart than an address space reaches is refused: their span does not fit the
arithmetic that looks for overlaps."""
import pytest

import block_sparse_attention_idx_b200 as msa
from test_tree_host import _rope


@pytest.mark.parametrize("kw", [
    dict(tokens=1 << 30, x_stride=1 << 39, y_stride=1 << 39, y=0x180000), dict(tokens=(1 << 31) - 1, x_stride=1 << 39),
    dict(tokens=(1 << 31) - 1, y_stride=1 << 39), dict(tokens=1 << 25, x_stride=1 << 37, y_stride=1 << 37, x_type=1, y_type=1)])
@pytest.mark.parametrize("fn", ["msa_rope_fwd", "msa_rope_bwd"])
def test_spans_past_the_address_space_are_refused(kw, fn):
    assert _rope(fn=fn, **kw) == msa.MSA_ERR_INVALID_ARG
