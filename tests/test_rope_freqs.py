"""YaRN frequencies against the pairs' turns counted one by one, and against values worked out by hand."""
import math

import pytest
import torch

import block_sparse_attention_idx_b200 as msa


def _by_turns(rot, base, factor, orig_len):
    """f_i = base^(-2 i / rot) kept up to the last pair that turns 32 times over orig_len, divided by factor from the first
    that turns at most once, mixed linearly in i between (from pair 0 where none turns 32 times; the pairs are counted
    past rot / 2, up to rot - 1)."""
    f = [base ** (-2 * i / rot) for i in range(rot)]
    turns = [orig_len * x / (2 * math.pi) for x in f]
    first_slow = next((i for i, t in enumerate(turns) if t <= 1), rot - 1)
    last_fast = max((i for i, t in enumerate(turns) if t >= 32), default=0)
    out = []
    for i in range(rot // 2):
        m = 1.0 if turns[i] <= 1 else 0.0 if turns[i] >= 32 else (i - last_fast) / (first_slow - last_fast)
        out.append(f[i] * (1 - m) + f[i] / factor * m)
    return torch.tensor(out, dtype=torch.float64)


@pytest.mark.parametrize("rot,base,factor,orig_len", [
    (128, 10000.0, 16.0, 4096), (64, 10000.0, 8.0, 131072), (128, 500000.0, 8.0, 8192), (32, 10000.0, 4.0, 32768),
    (16, 100.0, 2.0, 1000), (128, 10000.0, 32.0, 128), (64, 10000.0, 4.0, 12), (2, 10000.0, 4.0, 4096), (8, 1.5, 4.0, 512),
    (64, 10000.0, 4.0, 6), (64, 10000.0, 4.0, 1)])
def test_yarn_frequencies(rot, base, factor, orig_len):
    f, amp = msa.msa_rope_inv_freq(rot, base=base, scaling="yarn", factor=factor, orig_len=orig_len)
    assert torch.allclose(f, _by_turns(rot, base, factor, orig_len), rtol=1e-13, atol=0)
    assert amp == 0.1 * math.log(factor) + 1


def test_yarn_bounds_of_a_4096_token_model():
    """64 pairs, base 10000: pair i turns 4096 / (2 pi) 10000^(-i / 64) times, 36.7 times at i = 20 and 31.7 at 21, 1.004 at 45
    and 0.87 at 46. So 20 is the last kept, 46 the first divided, and 33 half way."""
    f, _ = msa.msa_rope_inv_freq(128, scaling="yarn", factor=16.0, orig_len=4096)
    plain, _ = msa.msa_rope_inv_freq(128)
    m = (1 - f / plain) / (1 - 1 / 16)
    want = ((torch.arange(64, dtype=torch.float64) - 20) / 26).clamp(0, 1)
    assert (m - want).abs().max() < 1e-14 * 16
    assert f[20] == plain[20] and m[21] > 0 and abs(float(m[33]) - 0.5) < 1e-13 and abs(float(f[46] * 16 / plain[46]) - 1) < 1e-15


def test_a_factor_of_one_changes_nothing():
    f, amp = msa.msa_rope_inv_freq(96, scaling="yarn", factor=1.0, orig_len=4096)
    plain, _ = msa.msa_rope_inv_freq(96)
    assert torch.allclose(f, plain, rtol=1e-15, atol=0) and amp == 1.0
