"""Selection for trees: the Top-k variant that ranks a row's 513 to 2048 blocks with one warp, which takes 16 rows an SM, and
what a sequence's selection and attention keep when the batch around it changes."""
import numpy as np
import pytest
import torch

import block_sparse_attention_idx_b200 as msa
from oracle import tree as otree
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN = float("nan")


def _rows():
    return 16 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("bk,topk,L", [(32, 16, 20000), (64, 16, 131071), (128, 5, 90000), (32, 1, 65536)])
def test_many_rows_of_up_to_2048_blocks(bk, topk, L):
    """Rows enough to fill the device: a warp a row, up to 64 candidates a lane."""
    T, H_kv = 64, 8
    B = -(-_rows() // (T * H_kv))
    assert 512 < -(-L // 256) * (256 // bk) <= 2048
    lens = [L - 37 * b for b in range(B)]
    c = Case(lens, T, H_q=H_kv, H_kv=H_kv, d=64, di=32, bk=bk, topk=topk, seed=81, N=L, n_nodes=[T] * (B - 1) + [T - 3])
    blocks, margin = c.select(want_margin=True)
    c.check_selection(blocks, margin, nodes=[0, T - 4, T - 1])


@pytest.mark.parametrize("lanes", [1, 15, 17])
def test_the_largest_maxima_in_few_lanes(lanes):
    """Lane l of the warp holds the maxima of blocks 4 l + {0 .. 3} + 128 j. With all large ones in `lanes` lanes, those
    lanes' candidates all pass the bound when there are no more than topk of them: up to 16 x 64 of the list's room."""
    T, H_kv, bk, topk, L = 64, 8, 32, 16, 2040 * 32
    B = -(-_rows() // (T * H_kv))
    c = Case([L] * B, T, H_q=H_kv, H_kv=H_kv, d=64, di=32, bk=bk, topk=topk, seed=82, N=L, kind="roots")
    blk = torch.arange(L // bk, device=DEV)
    high = (blk // 4) % 32 < lanes
    for b in range(B):  # the first element of a key decides, the queries all take it
        k = c.kip[c.table[b, :L // bk].long()]
        k[:, :, 0] = torch.where(high, 4.0, -4.0)[:, None].to(k.dtype)
        c.kip[c.table[b, :L // bk].long()] = k
    c.q_idx[..., 0] = 4.0
    c.q_idx[..., 1:] /= 16  # (2^-8 steps, times keys in 2^-4 steps: still exact)
    blocks, margin = c.select(want_margin=True)
    c.check_selection(blocks, margin, nodes=[0, 31, 63])
    assert high[blocks[..., :topk].long()].all()


def test_fewer_lanes_with_blocks_than_chosen_ones():
    """Short sequences in a long table: the variant is chosen by the table, most lanes hold no block."""
    T, H_kv, bk = 64, 8, 32
    B = max(-(-_rows() // (T * H_kv)), 7)
    lens = [0, 1, 31, 5 * 32, 64 * 32 - 1, 64 * 32, 128 * 32 + 7] + [3000] * (B - 7)
    c = Case(lens, T, H_q=H_kv, H_kv=H_kv, d=64, di=32, bk=bk, topk=16, seed=83, N=2048 * 32)
    blocks, margin = c.select(want_margin=True)
    c.check_selection(blocks, margin, nodes=[0, 63])


def _sub(c, keep):
    """The sequences `keep` of a case, over the same pools."""
    x = object.__new__(Case)
    x.__dict__.update(c.__dict__)
    at = torch.tensor(keep, device=DEV)
    x.dm = msa.MsaDims(len(keep), *[getattr(c.dm, f) for f in ("N", "H_q", "H_kv", "d", "d_idx", "block_k", "topk")])
    for f in ("table", "lens", "parents", "n_nodes", "q", "q_idx", "k", "v", "k_idx"):
        setattr(x, f, getattr(c, f)[at].contiguous())
    x.pages, x.tree = msa.MsaPages(x.table, x.lens), msa.MsaTree(x.parents, x.n_nodes)
    return x


@pytest.mark.parametrize("T,H_q,H_kv,d,bk", [(12, 64, 4, 128, 128), (40, 32, 1, 64, 32)])
def test_a_sequence_alone_and_in_other_batches(T, H_q, H_kv, d, bk):
    """Selection and margins do not depend on the batch, bit for bit. The attention's split of a sequence's keys does, by the
    other sequences' node counts: two results lie within twice the bound of one, 2 (2^-8 / (1 - 2^-8) + 3e-5) dev +
    4e-5 mag, where dev <= 2 mag."""
    lens = [1500, 300, 77, 4000, 0, 900]
    c = Case(lens, T, H_q=H_q, H_kv=H_kv, d=d, di=64, bk=bk, topk=16, seed=8, n_nodes=[T, T - 1, T, 1, T, 0])
    g = torch.Generator(device=DEV).manual_seed(85)
    for x in (c.q_idx, c.k_idx, c.kip):  # off the grid: sums that depend on their order
        x.copy_(torch.where(torch.isnan(x), x, torch.randn(x.shape, generator=g, device=DEV).to(x.dtype)))
    blocks, margin = c.select(want_margin=True)
    out, lse = c.attend(blocks, want_lse=True)
    for keep in ([0], [1], [2], [3], [4], [5], [3, 0], [5, 2, 1, 4], [1] * 7 + [0]):
        s = _sub(c, keep)
        b2, m2 = s.select(want_margin=True)
        assert torch.equal(b2, blocks[keep]) and torch.equal(m2, margin[keep])
        o2, l2 = s.attend(b2, want_lse=True)
        for i, b in enumerate(keep):
            nn = int(c.n_nodes[b])
            assert torch.equal(o2[i, nn:], out[b, nn:]) and torch.equal(l2[i, nn:], lse[b, nn:])
            for n in sorted({0, nn // 2, nn - 1}) if nn else []:
                K, V, _ = c.virtual(b, n)
                _, _, mag = otree.attend(c.od, c.q[b, n].cpu(), K, V, blocks[b, n].cpu().numpy())
                tol = 2 * (4 * (2.0 ** -8 / (1 - 2.0 ** -8) + 3e-5) + 4e-5) * mag
                assert (np.abs((o2[i, n] - out[b, n]).cpu().numpy()) <= tol).all()
            assert (l2[i, :nn] - lse[b, :nn]).abs().nan_to_num(0.0).max() <= 6e-5 if nn else True


@pytest.mark.parametrize("layout", [dict(H_q=8, H_kv=2, d=64, di=32, bk=32, topk=4), dict(H_q=16, H_kv=4, d=128, di=64, bk=128, topk=3),
                                    dict(H_q=4, H_kv=4, d=64, di=64, bk=64, topk=4)], ids=["bk32", "bk128", "bk64"])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_are_nan_do_not_count(layout, sign):
    """As in the oracle and the decode step: NaN keys in a block leave its other keys' maximum, a block of NaN keys has the
    maximum -inf, and so has everything for a NaN query; cached and drafted keys alike."""
    bk = layout["bk"]
    # a chain over a cache that ends two tokens before a block's end: node 1 fills it, node 2 opens the next
    c = Case([10 * bk - 2], 5, kind="chain", seed=87, **layout)
    c.q_idx[..., :4] = 4.0
    for x in (c.kip, c.k_idx):  # all scores around 64, or around -64
        x[..., :4] = torch.where(torch.isnan(x[..., :4]), x[..., :4], torch.full_like(x[..., :4], 4.0 * sign))
    c.kip[int(c.table[0, 2])] = NAN
    c.kip[int(c.table[0, 5]), :-1] = NAN
    c.kip[int(c.table[0, 5]), -1] = c.q_idx[0, 3, 0]  # what is left leads for node 3
    c.kip[int(c.table[0, 9]), :bk - 2] = NAN              # of the last block the drafted tokens' alone are numbers
    c.q_idx[0, 4, 0] = NAN
    for bad in (None, 0, 1):  # no, one and both of the drafted tokens that share the cache's last block
        if bad is not None:
            c.k_idx[0, bad] = NAN
        blocks = c.select().cpu().numpy()
        for n in range(5):
            K, V, KI = c.virtual(0, n)
            want, _, _, _ = otree.node_decode(c.od, c.q[0, n].cpu(), c.q_idx[0, n].cpu(), K, V, KI)
            assert (blocks[0, n] == want).all(), (bad, n, blocks[0, n], want)
    assert 5 in blocks[0, 3, 0] and 2 not in blocks[0, 3, 0]
    dm = msa.MsaDims(1, c.dm.N + 1, *[getattr(c.dm, f) for f in ("H_q", "H_kv", "d", "d_idx", "block_k", "topk")])
    dense = [torch.zeros(1, c.dm.N + 1, *p.shape[2:], dtype=torch.bfloat16, device=DEV) for p in (c.kp, c.vp, c.kip)]
    for n in range(5):  # the framework's decode step on the path
        for t, x in zip(dense, c.virtual(0, n)):
            t[0, :x.shape[0]] = x
        step = msa.msa_sparse_attn_decode(dm, c.lens + n + 1, c.q[0, n][None], c.q_idx[0, n][None], *dense)[1]
        assert (step[0].cpu().numpy() == blocks[0, n]).all(), n
