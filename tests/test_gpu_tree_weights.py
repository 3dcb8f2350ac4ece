"""The tree attention's weights sum to one whatever their rounding: the output is sum_j p_j (1 + e_j) v_j over
sum_j p_j (1 + e_j), |e_j| <= 2^-8 the rounding of a weight to bf16 for the product.

With o = sum_j w_j v_j the exact output, the error is sum_j w_j e_j (v_j - o) over 1 + sum_j w_j e_j: at most
2^-8 / (1 - 2^-8) of dev = sum_j w_j |v_j - o|. Keys split over CTAs are normalised part by part, o_p in place of o, and
merged with fp32 weights: as sum_p W_p |o_p - o| <= dev, the bound there is twice that. A value common to all keys is
therefore kept, to the fp32 roundings: at most 128 additions in a row to either sum, 2^-24 each, and as many
accumulations of a product of 16, taken as 2^-22 each: 4e-5 of sum_j w_j |v_j| with the exponentials' own error (a part
of a weight, so part of dev) left aside. Logits are good to 3e-5, in the weights, dev again."""
import numpy as np
import pytest
import torch

import block_sparse_attention_idx_b200 as msa
from oracle import tree as otree
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu

DEV = "cuda"
I32 = torch.int32


def _set_v(c, f):
    """V = f(tokens) wherever a token is (NaN elsewhere, as Case left it)."""
    for x in (c.v, c.vp):
        x.copy_(torch.where(torch.isnan(x), x, f(x).to(x.dtype)))


def _exact(c, blocks, b, n):
    """Output, weighted mean of |v - out| and of |v| of a node, in 64 bits."""
    K, V, _ = c.virtual(b, n)
    lists = blocks[b, n].cpu().numpy()
    o, _, mag = otree.attend(c.od, c.q[b, n].cpu(), K, V, lists)
    dev = np.zeros_like(o)
    G = c.od.H_q // c.od.H_kv
    for h in range(c.od.H_q):  # |v - o| has its own o per output element
        ids = sorted({int(x) for x in lists[h // G] if x >= 0})
        J = [j for x in ids for j in range(x * c.od.block_k, min((x + 1) * c.od.block_k, K.shape[0]))]
        z = K[J, h // G].double().numpy() @ c.q[b, n, h].cpu().double().numpy() / c.od.d ** 0.5
        w = np.exp(z - z.max())
        dev[h] = (w / w.sum()) @ np.abs(V[J, h // G].double().numpy() - o[h])
    return o, dev, mag


CASES = [dict(lens=[150, 31, 64, 0], T=5, H_q=8, H_kv=2, d=64, di=32, bk=32, topk=4),
         dict(lens=[700, 1024], T=3, H_q=64, H_kv=4, d=128, di=64, bk=128, topk=5),
         dict(lens=[640], T=9, H_q=32, H_kv=1, d=64, di=32, bk=64, topk=16),
         dict(lens=[900, 77], T=1, H_q=16, H_kv=8, d=128, di=32, bk=32, topk=16)]


@pytest.mark.parametrize("case", CASES, ids=lambda x: f"d{x['d']}-bk{x['bk']}-T{x['T']}")
def test_values_that_all_keys_share_come_out_as_they_are(case):
    c = Case(seed=61, **case)
    col = torch.linspace(0.5, 2.0, c.dm.d, device=DEV).to(torch.bfloat16)
    _set_v(c, lambda x: col.expand(x.shape))
    out, _ = c.attend(c.select())
    assert (out.double() / col.double() - 1).abs().max() <= 4e-5
    half, _ = c.attend(c.select(), out_dtype=torch.bfloat16)
    assert torch.equal(half, col.expand(half.shape))


@pytest.mark.parametrize("case", CASES, ids=lambda x: f"d{x['d']}-bk{x['bk']}-T{x['T']}")
def test_an_offset_of_the_values_adds_no_error(case):
    """V around 64, its deviations around 1: the error follows the deviations."""
    c = Case(seed=62, **case)
    _set_v(c, lambda x: x.float() + 64)
    blocks = c.select()
    out, _ = c.attend(blocks)
    for b in range(c.dm.B):
        for n in range(int(c.n_nodes[b])):
            o, dev, mag = _exact(c, blocks, b, n)
            tol = 2 * (2.0 ** -8 / (1 - 2.0 ** -8) + 3e-5) * dev + 4e-5 * mag
            err = np.abs(out[b, n].double().cpu().numpy() - o)
            assert (err <= tol).all(), (b, n, (err / tol).max())


def test_a_late_key_that_leads_without_raising_the_maximum():
    """The lazily raised maximum leaves a leading key the weight 196.6, which bf16 rounds by 2e-3: the row is that key's
    value all the same. One head whose query picks the first element of a key, d = 64, so that a logit is K_0 / 8."""
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count  # items enough that none is split
    c = Case([64] * B, 1, H_q=1, H_kv=1, d=64, di=32, bk=32, topk=2, seed=63)
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.k.zero_()  # the drafted token's own logit is 0: the first tile's maximum
    c.kp.zero_()
    c.kp[:, :, 0, 0] = -1024.0  # weight e^-128
    c.kp[c.table[:, 1].long(), 7, 0, 0] = 42.25  # 2^(42.25 / 8 log2 e) = 196.6
    blocks = torch.tensor([0, 1, 2], dtype=I32, device=DEV).expand(B, 1, 1, 3).contiguous()
    out, lse = c.attend(blocks, want_lse=True)
    assert (lse.double() - np.logaddexp(0.0, 42.25 / 8)).abs().max() <= 3e-5
    for b in (0, 1, B - 1):
        o, dev, mag = _exact(c, blocks, b, 0)
        err = np.abs(out[b, 0].double().cpu().numpy() - o)
        assert (err <= (2.0 ** -8 / (1 - 2.0 ** -8) + 3e-5) * dev + 4e-5 * mag).all()


def test_one_node_is_as_exact_as_the_decode_step():
    """Both normalise by the sum of the rounded weights: against 64 bits, values around 64, the paged step stays within
    the decode step's bound (twice it where its keys are split)."""
    lens = [700, 33, 511, 1, 1024]
    c = Case(lens, 1, H_q=64, H_kv=4, d=128, di=64, bk=128, topk=16, seed=64, N=1100)
    _set_v(c, lambda x: x.float() + 64)
    blocks = c.select()
    out, _ = c.attend(blocks)
    N = 1101
    dense = [torch.zeros(len(lens), N, *p.shape[2:], dtype=torch.bfloat16, device=DEV) for p in (c.kp, c.vp, c.kip)]
    for b, n in enumerate(lens):
        for t, p, x in zip(dense, (c.kp, c.vp, c.kip), (c.k, c.v, c.k_idx)):
            t[b, :n + 1] = torch.cat([otree.gather_pages(p, c.table[b], n), x[b]])
    dm = msa.MsaDims(len(lens), N, 64, 4, 128, 64, 128, 16)
    step, _ = msa.msa_sparse_attn_decode(dm, c.lens + 1, c.q[:, 0].contiguous(), c.q_idx[:, 0].contiguous(), *dense)
    for b in range(len(lens)):
        o, dev, mag = _exact(c, blocks, b, 0)
        one = (2.0 ** -8 / (1 - 2.0 ** -8) + 3e-5) * dev
        for got, tol in ((out[b, 0], 2 * one + 4e-5 * mag), (step[b], 2 * one + 4e-5 * mag)):
            assert (np.abs(got.double().cpu().numpy() - o) <= tol).all()
