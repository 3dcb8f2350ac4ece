"""Rotary angles of any position. A pair (1, 0) comes out as (cos, sin) of its angle, exactly as the kernel has them, and is
compared with the angle reduced in integers (the frequency over 2 pi as a fraction of 2^-260, times the position): the
documented bound is 3e-7. It holds an angle's rounding to fp32 in half turns (2^-25 pi = 9.4e-8) and a unit in the last
place of sincospi (at most 2^-23 = 1.2e-7)."""
import math
from fractions import Fraction

import pytest
import torch

import block_sparse_attention_idx_b200 as msa

pytestmark = pytest.mark.gpu

DEV = "cuda"
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")
SHIFT = 260


def _cos_sin(positions, freqs):
    """[tokens, frequencies] cosines and sines in fp64, angles reduced without a rounding."""
    turns = [round(Fraction(f) / (2 * PI) * (1 << SHIFT)) for f in freqs]
    rows = [[math.ldexp((p * w & ((1 << SHIFT) - 1)) >> (SHIFT - 64), -64) * (2 * math.pi) for w in turns] for p in positions]
    a = torch.tensor(rows, dtype=torch.float64)
    return a.cos(), a.sin()


def _check(positions, f, interleaved=False, back=False):
    r = 2 * f.numel()
    x = torch.zeros(len(positions), 1, 128, device=DEV)
    x[..., 0:r:2 if interleaved else 1][..., :r // 2] = 1.0
    pos = torch.tensor(positions, dtype=torch.int64).to(torch.int32).to(DEV)
    turn = msa.msa_rope_bwd if back else msa.msa_rope_fwd
    y, = turn([x], [(f.to(DEV), 1.0)], pos, interleaved=interleaved)
    y = y[:, 0].double().cpu()
    a, b = (y[:, 0:r:2], y[:, 1:r:2]) if interleaved else (y[:, :r // 2], y[:, r // 2:r])
    c, s = _cos_sin(positions, f.tolist())
    assert (a - c).abs().max() <= 3e-7
    assert (b - (-s if back else s)).abs().max() <= 3e-7


def _positions(n, lo, hi, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi, (n,), generator=g, dtype=torch.int64).tolist()


@pytest.mark.parametrize("scaling,kw", [(None, {}), ("linear", dict(factor=8.0)), ("yarn", dict(factor=16.0, orig_len=4096))])
@pytest.mark.parametrize("lo,hi", [(0, 4096), (1 << 19, 1 << 20), (1 << 30, (1 << 31) - 1), (-(1 << 31), -(1 << 30))])
def test_cosines_and_sines_of_near_and_far_positions(lo, hi, scaling, kw):
    f, _ = msa.msa_rope_inv_freq(128, scaling=scaling, **kw)
    _check(_positions(3000, lo, hi, 5) + [lo, hi], f)


@pytest.mark.parametrize("interleaved,back", [(False, True), (True, False), (True, True)])
def test_layouts_and_the_gradient_at_far_positions(interleaved, back):
    f, _ = msa.msa_rope_inv_freq(96)
    _check(_positions(500, -(1 << 31), 1 << 31, 6), f, interleaved, back)


@pytest.mark.parametrize("top", [1.0, 1000.5, 2.0 ** 16.9])
def test_frequencies_up_to_the_documented_product(top):
    """|position * inv_freq| < 2^48, the largest too."""
    f = torch.logspace(0, -3, 32, dtype=torch.float64) * top * (1 - 2.0 ** -20)
    _check(_positions(500, -(1 << 31), 1 << 31, 7) + [-(1 << 31), (1 << 31) - 1, 0, 1, -1], f)
    _check([3, 1000003], -f)
