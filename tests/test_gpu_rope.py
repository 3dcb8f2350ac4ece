"""Rotary positions against a float64 evaluation, their gradient against the formula and differences.

cos and sin are fp32 values of an angle reduced in 64 bits: absolute error at most 3e-7. With |x| the
pair's norm, a rotated element is off by amp |x| (3e-7 + 2 * 2^-24) from them and the two fp32 products, and
by half a step of the output type: 2^-24 (fp32) or 2^-8 (bf16) of the value. The tests' tolerance is
4.5e-7 amp |x| plus that half step."""
import math

import pytest
import torch

import block_sparse_attention_idx_b200 as msa
from oracle import tree as otree

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _pair_norm(x, rot, interleaved, amp):
    """amp * norm of each element's pair (0 for elements that are copied)."""
    z = torch.zeros(x.shape, dtype=torch.float64)
    y = x.double().cpu()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    n = (y[..., a] ** 2 + y[..., b] ** 2).sqrt() * amp
    z[..., a], z[..., b] = n, n
    return z


def _check(x, y, f, amp, pos, interleaved, back=False):
    want = torch.from_numpy(otree.rope(x, f, amp, pos.cpu(), interleaved, back))
    half = torch.finfo(y.dtype).eps / 2
    tol = 4.5e-7 * _pair_norm(x, 2 * f.numel(), interleaved, amp) * (1 + half) + half * want.abs()
    err = (y.double().cpu() - want).abs()
    assert (err <= tol).all(), f"max excess {(err - tol).max():.3e}"


def _x(g, *s, dtype=BF):
    return torch.randn(*s, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("tokens,heads,dim,rot", [
    (1, 1, 32, 32), (1, 64, 128, 128), (3, 4, 64, 64), (7, 5, 128, 64), (33, 3, 128, 96), (17, 2, 64, 2),
    (5, 7, 128, 126), (9, 1, 32, 12), (4, 3, 64, 40), (2, 16, 128, 16), (130, 2, 32, 8),
])
def test_rope_matches_float64(tokens, heads, dim, rot, dtype, out, interleaved):
    g = torch.Generator(device=DEV).manual_seed(tokens * 1000 + rot)
    x = _x(g, tokens, heads, dim, dtype=dtype)
    f, amp = msa.msa_rope_inv_freq(rot, device=DEV)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device=DEV, dtype=torch.int32)
    y, = msa.msa_rope_fwd([x], [(f, 1.25)], pos, interleaved=interleaved, out_dtype=out)
    assert y.dtype == out
    _check(x, y, f, 1.25, pos, interleaved)
    dx, = msa.msa_rope_bwd([x], [(f, amp)], pos, interleaved=interleaved, out_dtype=out)
    _check(x, dx, f, amp, pos, interleaved, back=True)


@pytest.mark.parametrize("scaling,kw", [(None, {}), ("linear", dict(factor=8.0)), ("ntk", dict(factor=4.0)),
                                        ("yarn", dict(factor=16.0, orig_len=4096))])
def test_four_tensors_in_one_call_far_and_negative_positions(scaling, kw):
    g = torch.Generator(device=DEV).manual_seed(5)
    n = 37
    xs = [_x(g, n, 16, 128), _x(g, n, 2, 128), _x(g, n, 2, 64), _x(g, n, 1, 64)]
    f, amp = msa.msa_rope_inv_freq(128, scaling=scaling, device=DEV, **kw)
    fi, ampi = msa.msa_rope_inv_freq(32, scaling=scaling, device=DEV, **kw)
    freqs = [(f, amp), (f, amp), (fi, ampi), (fi, ampi)]
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (n,), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    pos[:4] = torch.tensor([0, 1, -1, 2 ** 31 - 1], dtype=torch.int32)
    ys = msa.msa_rope_fwd(xs, freqs, pos)
    # at 2^31 a frequency's own rounding (2^-53) moves the angle by 2e-7 rad times f: positions up to 2^24 hold
    # the ordinary tolerance, the others three times that
    for x, y, (ff, a) in zip(xs, ys, freqs):
        want = torch.from_numpy(otree.rope(x, ff, a, pos.cpu(), False))
        tol = (1.4e-6 + 2 ** -31) * _pair_norm(x, 2 * ff.numel(), False, a) * 1.01 + 2 ** -8 * want.abs()
        assert ((y.double().cpu() - want).abs() <= tol).all()


def test_default_positions_are_token_indexes_and_in_place_equals_out_of_place():
    g = torch.Generator(device=DEV).manual_seed(6)
    x = _x(g, 2, 50, 4, 64)
    f, amp = msa.msa_rope_inv_freq(48, device=DEV)
    want, = msa.msa_rope_fwd([x], [(f, amp)], torch.arange(100, device=DEV, dtype=torch.int32).view(2, 50))
    got, = msa.msa_rope_fwd([x], [(f, amp)])
    assert torch.equal(want, got)
    buf = x.clone()
    same, = msa.msa_rope_fwd([buf], [(f, amp)], outs=[buf])
    assert same is buf and torch.equal(buf, want)


@pytest.mark.parametrize("tokens", [1, 300, 9000])
def test_slices_of_a_projection_are_rotated_in_place(tokens):
    """Q and K as column slices of one [tokens, (H_q + 2 H_kv) d] buffer: V's columns stay as they were."""
    g = torch.Generator(device=DEV).manual_seed(tokens)
    qkv = _x(g, tokens, 12, 64)
    ref = qkv.clone()
    f, amp = msa.msa_rope_inv_freq(64, device=DEV)
    q, k = qkv[:, :8], qkv[:, 8:10]
    msa.msa_rope_fwd([q, k], [(f, amp)] * 2, outs=[q, k])
    wq, wk = msa.msa_rope_fwd([ref[:, :8].contiguous(), ref[:, 8:10].contiguous()], [(f, amp)] * 2)
    assert torch.equal(qkv[:, :8], wq) and torch.equal(qkv[:, 8:10], wk) and torch.equal(qkv[:, 10:], ref[:, 10:])


def test_large_launch_slices_agree_with_small_ones():
    """The work split depends on the number of tokens; the values do not."""
    g = torch.Generator(device=DEV).manual_seed(8)
    x = _x(g, 20000, 64, 128)
    f, amp = msa.msa_rope_inv_freq(128, device=DEV)
    pos = torch.randint(0, 1 << 20, (20000,), generator=g, device=DEV, dtype=torch.int32)
    y, = msa.msa_rope_fwd([x], [(f, amp)], pos)
    for lo, hi in ((0, 1), (777, 1010), (19990, 20000)):
        z, = msa.msa_rope_fwd([x[lo:hi]], [(f, amp)], pos[lo:hi].clone())
        assert torch.equal(y[lo:hi], z)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_is_the_transpose_and_matches_differences(interleaved):
    """<dy, R x> = <R^T dy, x>; and the map is linear, so that a difference quotient of <dy, R x> along any u
    equals <R^T dy, u> up to the fp32 roundings (2^-24 each, on sums of 6144 products of unit scale)."""
    g = torch.Generator(device=DEV).manual_seed(9)
    x, dy, u = (_x(g, 16, 3, 128, dtype=F32) for _ in range(3))
    f, _ = msa.msa_rope_inv_freq(96, device=DEV)
    fr = [(f, 1.5)]
    pos = torch.randint(0, 100000, (16,), generator=g, device=DEV, dtype=torch.int32)
    R = lambda t: msa.msa_rope_fwd([t], fr, pos, interleaved=interleaved)[0].double()  # noqa: E731
    dx = msa.msa_rope_bwd([dy], fr, pos, interleaved=interleaved)[0].double()
    d = dy.double()
    tol = 1e-6 * 1.5 * x.numel() ** 0.5 * 4
    assert abs((d * R(x)).sum() - (dx * x.double()).sum()) < tol
    h = 0.5
    diff = ((d * R(x + h * u)).sum() - (d * R(x - h * u)).sum()) / (2 * h)
    assert abs(diff - (dx * u.double()).sum()) < 4 * tol


def test_empty_strange_values_and_streams():
    f, amp = msa.msa_rope_inv_freq(64, device=DEV)
    e, = msa.msa_rope_fwd([torch.empty(0, 4, 64, dtype=BF, device=DEV)], [(f, amp)])
    assert e.shape == (0, 4, 64)
    x = torch.zeros(2, 1, 64, dtype=BF, device=DEV)
    x[0, 0, 3], x[0, 0, 40] = math.inf, math.nan
    y, = msa.msa_rope_fwd([x], [(f, amp)], torch.tensor([5, 6], dtype=torch.int32, device=DEV))
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, [3, 35, 8, 40]] = True  # the pairs (3, 35) and (8, 40) alone
    assert torch.equal(bad, want)
    s = torch.cuda.Stream()
    x = torch.randn(64, 4, 64, device=DEV).to(BF)
    s.wait_stream(torch.cuda.current_stream())
    a, = msa.msa_rope_fwd([x], [(f, amp)], stream=s)
    s.synchronize()
    assert torch.equal(a, msa.msa_rope_fwd([x], [(f, amp)])[0])


def test_captured_and_replayed():
    f, amp = msa.msa_rope_inv_freq(64, device=DEV)
    x = torch.randn(100, 4, 64, device=DEV).to(BF)
    pos = torch.zeros(100, dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    msa.msa_rope_fwd([x], [(f, amp)], pos, outs=[out])
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        msa.msa_rope_fwd([x], [(f, amp)], pos, outs=[out])
    pos += 17
    x.neg_()
    gr.replay()
    assert torch.equal(out, msa.msa_rope_fwd([x], [(f, amp)], pos)[0])
