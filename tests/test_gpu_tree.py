"""Drafted-token trees over a paged cache: selection and attention of every node against the oracle's decode
step on the node's virtual sequence (the cached tokens, its ancestors and itself).

Index vectors lie on a grid of 1/16 with magnitude up to 4: every product and sum of a score is exact in fp32
in any order, so that block lists (ties included) have to be equal.

Attention tolerance. The product takes p_j as bf16, p_j (1 + e_j) with |e_j| <= 2^-8, and the output is normalised
by the sum of the unrounded p_j, as the prefill kernel's is: with w_j = p_j / sum p, the output is
sum_j w_j (1 + e_j) v_j, so that |error| <= 2^-8 sum_j w_j |v_j|. (An earlier kernel normalised by the rounded
weights' sum, error sum_j w_j e_j (v_j - o) / (1 + ...), and was tested against that smaller bound; the unrounded
sum saves a third of the instructions of a weight.) The logits (fp32 accumulation over d <= 128 products,
|q.k| scale < 16) and the base-2 exponential are good to 3e-5 relative, in the weights again. A bf16 output adds
half a step, 2^-8 of the value. LSE: 3e-5."""
import numpy as np
import pytest
import torch

import block_sparse_attention_idx_b200 as msa
import oracle
from oracle import tree as otree

pytestmark = pytest.mark.gpu

DEV = "cuda"
I32 = torch.int32
NAN = float("nan")


def _grid(g, *s):
    return (torch.randn(*s, generator=g, device=DEV).clamp(-4, 4) * 16).round().div(16).to(torch.bfloat16)


def _bf(g, *s):
    return torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)


def _parents(kind, B, T, g):
    n = torch.arange(T, device=DEV)
    if kind == "chain":
        p = (n - 1).expand(B, T)
    elif kind == "roots":
        p = torch.full((B, T), -1, device=DEV)
    else:
        p = n - 1 - (torch.rand(B, T, generator=g, device=DEV) * 4).long()
    return p.clamp(min=-1).to(I32).contiguous()


class Case:
    """A batch of trees over a shuffled pool. Everything no node may see is NaN: unused pages, the last page
    behind the last token, drafted rows of absent nodes."""

    def __init__(self, lens, T, H_q=8, H_kv=2, d=64, di=32, bk=32, topk=4, kind="random", n_nodes=None, seed=0, N=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        B = len(lens)
        N = max(max(lens), 1) + 7 if N is None else N
        cols = -(-N // bk)
        self.od = oracle.Dims(B, N, H_q, H_kv, d, di, bk, topk)
        self.dm = msa.MsaDims(B, N, H_q, H_kv, d, di, bk, topk)
        pages = B * cols + 3
        self.table = torch.randperm(pages, generator=g, device=DEV)[:B * cols].view(B, cols).to(I32)
        self.lens = torch.tensor(lens, dtype=I32, device=DEV)
        self.parents = _parents(kind, B, T, g)
        nn = [T] * B if n_nodes is None else n_nodes
        self.n_nodes = torch.tensor(nn, dtype=I32, device=DEV)
        self.q, self.q_idx = _bf(g, B, T, H_q, d), _grid(g, B, T, H_kv, di)
        self.k, self.v, self.k_idx = _bf(g, B, T, H_kv, d), _bf(g, B, T, H_kv, d), _grid(g, B, T, di)
        self.kp, self.vp, self.kip = _bf(g, pages, bk, H_kv, d), _bf(g, pages, bk, H_kv, d), _grid(g, pages, bk, di)
        used = torch.zeros(pages, bk, dtype=torch.bool, device=DEV)
        for b in range(B):
            pos = torch.arange(lens[b], device=DEV)
            used[self.table[b].long()[pos // bk], pos % bk] = True
            for x in (self.q, self.q_idx, self.k, self.v, self.k_idx):
                x[b, nn[b]:] = NAN
        for p in (self.kp, self.vp, self.kip):
            p[~used] = NAN
        self.pages, self.tree = msa.MsaPages(self.table, self.lens), msa.MsaTree(self.parents, self.n_nodes)

    def select(self, **kw):
        return msa.msa_tree_index_topk(self.dm, self.pages, self.tree, self.q_idx, self.k_idx, self.kip, **kw)

    def attend(self, blocks, **kw):
        return msa.msa_tree_sparse_attn(self.dm, self.pages, self.tree, self.q, self.k, self.v, self.kp, self.vp, blocks, **kw)

    def virtual(self, b, n):
        """K, V, K_idx of node n's virtual sequence."""
        up, L = otree.path(self.parents[b], n), int(self.lens[b])
        return tuple(torch.cat([otree.gather_pages(p, self.table[b], L), x[b, up]]).cpu()
                     for p, x in ((self.kp, self.k), (self.vp, self.v), (self.kip, self.k_idx)))

    def check_selection(self, blocks, margin, nodes=None):
        T, k = self.parents.shape[1], self.dm.topk
        blocks, margin = blocks.cpu().numpy(), margin.cpu().numpy()
        for b in range(self.dm.B):
            nn = int(self.n_nodes[b])
            for n in range(T) if nodes is None else nodes:
                if n >= nn:
                    assert (blocks[b, n] == -1).all() and np.isposinf(margin[b, n]).all()
                    continue
                K, V, KI = self.virtual(b, n)
                want, m, _, _ = otree.node_decode(self.od, self.q[b, n].cpu(), self.q_idx[b, n].cpu(), K, V, KI)
                assert (blocks[b, n] == want).all(), (b, n, blocks[b, n], want)
                assert np.array_equal(np.isinf(m), np.isinf(margin[b, n]))
                f = np.isfinite(m)
                # the difference of two exact maxima, scaled: two roundings
                assert (np.abs(margin[b, n][f] - m[f]) <= 3 * 2.0 ** -24 * np.abs(m[f])).all()

    def check_attention(self, blocks, out, lse, nodes=None):
        T = self.parents.shape[1]
        lists = blocks.cpu().numpy()
        half = torch.finfo(out.dtype).eps / 2 if out.dtype == torch.bfloat16 else 2.0 ** -23
        got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.isfinite(got).all()
        for b in range(self.dm.B):
            nn = int(self.n_nodes[b])
            for n in range(T) if nodes is None else nodes:
                if n >= nn:
                    assert (got[b, n] == 0).all() and np.isneginf(glse[b, n]).all()
                    continue
                K, V, _ = self.virtual(b, n)
                o, l, mag = otree.attend(self.od, self.q[b, n].cpu(), K, V, lists[b, n])
                tol = (2.0 ** -8 + 3e-5) * mag * (1 + half) + half * np.abs(o) + 1e-6
                assert (np.abs(got[b, n] - o) <= tol).all(), (b, n, np.abs(got[b, n] - o).max())
                f = np.isfinite(l)
                assert np.array_equal(f, np.isfinite(glse[b, n]))
                assert (np.abs(glse[b, n][f] - l[f]) <= 3e-5).all()


LAYOUTS = [
    dict(H_q=8, H_kv=2, d=64, di=32, bk=32, topk=4), dict(H_q=64, H_kv=4, d=128, di=64, bk=128, topk=16),
    dict(H_q=1, H_kv=1, d=64, di=64, bk=64, topk=1), dict(H_q=8, H_kv=8, d=128, di=32, bk=32, topk=16),
    dict(H_q=32, H_kv=1, d=64, di=32, bk=128, topk=2), dict(H_q=16, H_kv=8, d=128, di=64, bk=64, topk=7),
    dict(H_q=64, H_kv=2, d=128, di=32, bk=64, topk=5),
]


def _run(c, nodes=None, **kw):
    blocks, margin = c.select(want_margin=True)
    c.check_selection(blocks, margin, nodes)
    out, lse = c.attend(blocks, want_lse=True, **kw)
    c.check_attention(blocks, out, lse, nodes)
    return blocks, out, lse


@pytest.mark.parametrize("layout", LAYOUTS, ids=lambda x: f"G{x['H_q'] // x['H_kv']}-{x['H_kv']}x{x['d']}-bk{x['bk']}-k{x['topk']}")
@pytest.mark.parametrize("T", [1, 5, 17])
def test_tree_matches_decode_on_the_virtual_sequences(layout, T):
    bk = layout["bk"]
    lens = [0, 1, bk - 1, bk, bk + 1, 3 * bk - 2, 9 * bk + 5]
    n_nodes = [T, max(1, T - 1), T, (T + 1) // 2, 0, T, T]
    _run(Case(lens, T, n_nodes=n_nodes, seed=T + bk, **layout))


@pytest.mark.parametrize("kind", ["chain", "roots", "random"])
@pytest.mark.parametrize("layout", [LAYOUTS[0], LAYOUTS[1], LAYOUTS[3]], ids=["bk32", "bk128", "heads8"])
def test_wide_and_deep_trees(layout, kind):
    """64 nodes: paths that leave the cache's last block behind and cross one or two of their own."""
    bk = layout["bk"]
    c = Case([0, 2 * bk - 3, 7 * bk], 64, kind=kind, n_nodes=[64, 63, 33], seed=11, **layout)
    _run(c, nodes=[0, 1, 30, 31, 32, 33, 62, 63])


def test_single_token_equals_the_decode_step_bit_for_bit_in_selection():
    """T = 1 against the framework's own decode over dense caches that already hold the new token."""
    lens = [700, 33, 511, 1, 1024]
    c = Case(lens, 1, H_q=64, H_kv=4, d=128, di=64, bk=128, topk=16, seed=3, N=1100)
    blocks, margin = c.select(want_margin=True)
    out, lse = c.attend(blocks, want_lse=True)
    N = 1101
    dense = [torch.zeros(len(lens), N, *p.shape[2:], dtype=torch.bfloat16, device=DEV) for p in (c.kp, c.vp, c.kip)]
    for b, n in enumerate(lens):
        for t, p, x in zip(dense, (c.kp, c.vp, c.kip), (c.k, c.v, c.k_idx)):
            t[b, :n + 1] = torch.cat([otree.gather_pages(p, c.table[b], n), x[b]])
    dm = msa.MsaDims(len(lens), N, 64, 4, 128, 64, 128, 16)
    o2, b2, m2 = msa.msa_sparse_attn_decode(dm, c.lens + 1, c.q[:, 0].contiguous(), c.q_idx[:, 0].contiguous(), *dense,
                                            want_margin=True)
    assert torch.equal(blocks[:, 0], b2) and torch.equal(margin[:, 0], m2)
    # both round P to bf16, against other maxima: twice the one-sided bound on unit-scale values
    assert (out[:, 0] - o2).abs().max() < 2 * 2.0 ** -8 * 4


@pytest.mark.parametrize("T,H_q", [(3, 8), (64, 64)])
def test_long_contexts_many_tiles(T, H_q):
    c = Case([20011, 8192, 16383], T, H_q=H_q, H_kv=4, d=128, di=64, bk=128, topk=16, seed=7, n_nodes=[T, T - 1, T])
    _run(c, nodes=[0, T - 2, T - 1], out_dtype=torch.bfloat16)


def test_ties_go_to_the_lowest_block():
    c = Case([40 * 32 + 3, 70 * 32], 6, topk=5, seed=1)
    c.kip[:] = torch.where(torch.isnan(c.kip), c.kip, torch.ones_like(c.kip))
    c.k_idx[:] = 1.0
    blocks, margin = c.select(want_margin=True)
    c.check_selection(blocks, margin)
    assert (margin == 0).all() and (blocks[..., :5] == torch.arange(5, device=DEV)).all()


def test_lists_with_holes_duplicates_and_empty_rows():
    """Any list is attended as the set of its ids: without the local block a node does not see itself, and an
    empty list gives 0 and -inf."""
    c = Case([5 * 32 + 9, 31], 7, seed=2, kind="chain")
    lists = torch.full((2, 7, 2, 5), -1, dtype=I32, device=DEV)
    lists[0, 0, 0] = torch.tensor([3, 3, -1, 0, 3])
    lists[0, 1, 1] = torch.tensor([-1, -1, 5, -1, -1])
    lists[0, 2, :, 2] = 4
    lists[0, 6, 0] = torch.tensor([5, 4, 3, 2, 1])
    lists[1, 3, 0, 0], lists[1, 6, 1, 4] = 1, 0
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = c.attend(lists, want_lse=True, out_dtype=dtype)
        c.check_attention(lists, out, lse)
    assert torch.isneginf(lse[0, 0, 4:]).all() and (out[1, 0] == 0).all()


def test_a_growing_maximum_rescales_what_was_summed():
    """Keys whose logits climb tile by tile: every tile raises the running maximum by more than 2^8."""
    c = Case([900], 2, H_q=16, H_kv=1, d=64, di=32, bk=128, topk=8, seed=4)
    blocks = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -1], dtype=I32, device=DEV).expand(1, 2, 1, 9).contiguous()
    for p in range(900 // 128 + 1):
        x = c.kp[int(c.table[0, p])]
        x[~torch.isnan(x)] *= 2.0 ** (p / 2)
    out, lse = c.attend(blocks, want_lse=True)
    K, V, _ = c.virtual(0, 0)
    o, l, mag = otree.attend(c.od, c.q[0, 0].cpu(), K, V, blocks[0, 0].cpu().numpy())
    # logits reach |60|: fp32 logits to 60 * 128 * 2^-24, weights to that relative
    assert (np.abs(out[0, 0].double().cpu().numpy() - o) <= (2.0 ** -8 + 5e-4) * mag + 1e-5).all()
    assert np.abs(lse[0, 0].double().cpu().numpy() - l).max() < 5e-4


def test_out_of_range_entries_are_read_as_documented_and_reported():
    c = Case([100, 64, 90], 4, seed=5, kind="chain")
    ws = msa.tree_workspace(msa.MSA_OP_TREE_INDEX_TOPK, c.dm, 4, DEV)
    wa = msa.tree_workspace(msa.MSA_OP_TREE_ATTN, c.dm, 4, DEV)

    def both():
        for p in (c.kp, c.vp, c.kip):
            p[torch.isnan(p)] = 0.5
        blocks = c.select(ws=ws)
        st = msa.msa_get_device_status(ws)
        out, lse = c.attend(blocks, want_lse=True, ws=wa)
        return blocks, out, lse, st, msa.msa_get_device_status(wa)

    for x in (c.q, c.q_idx, c.k, c.v, c.k_idx):
        x[torch.isnan(x)] = 0.25
    good = both()
    assert good[3:] == (msa.MSA_OK, msa.MSA_OK)
    c.parents[1, 2] = 2  # its own parent: read as -1
    bad = both()
    assert bad[3:] == (msa.MSA_ERR_DEVICE_CHECK,) * 2
    c.parents[1, 2] = -1
    again = both()
    assert again[3:] == (msa.MSA_OK, msa.MSA_OK) and all(torch.equal(x, y) for x, y in zip(bad[:3], again[:3]))
    c.lens[0], c.n_nodes[1] = c.dm.N + 50, 9  # clamped to N and T
    bad = both()
    assert bad[3:] == (msa.MSA_ERR_DEVICE_CHECK,) * 2
    c.lens[0], c.n_nodes[1] = c.dm.N, 4
    again = both()
    assert again[3:] == (msa.MSA_OK, msa.MSA_OK) and all(torch.equal(x, y) for x, y in zip(bad[:3], again[:3]))
    keep = c.table.clone()
    c.table[2, 1] = 1 << 30  # read as page 0
    bad = both()
    assert bad[3] == msa.MSA_ERR_DEVICE_CHECK
    c.table[2, 1] = 0
    again = both()
    assert again[3] == msa.MSA_OK and all(torch.equal(x, y) for x, y in zip(bad[:3], again[:3]))
    c.table.copy_(keep)
    blocks = c.select(ws=ws)
    wrong = blocks.clone()
    wrong[0, 0, 0, 0], wrong[0, 1, 0, 0] = -2, 1 << 20  # read as -1
    o1 = c.attend(wrong, ws=wa)[0]
    assert msa.msa_get_device_status(wa) == msa.MSA_ERR_DEVICE_CHECK
    wrong[0, 0, 0, 0], wrong[0, 1, 0, 0] = -1, -1
    o2 = c.attend(wrong, ws=wa)[0]
    assert msa.msa_get_device_status(wa) == msa.MSA_OK and torch.equal(o1, o2)


def test_results_do_not_depend_on_the_batch_or_repeat():
    c = Case([1500, 300, 77, 4000], 12, H_q=64, H_kv=4, d=128, di=64, bk=128, topk=16, seed=8)
    b1, m1 = c.select(want_margin=True)
    o1, l1 = c.attend(b1, want_lse=True)
    for _ in range(3):
        b2, m2 = c.select(want_margin=True)
        o2, l2 = c.attend(b1, want_lse=True)
        assert torch.equal(b1, b2) and torch.equal(m1, m2) and torch.equal(o1, o2) and torch.equal(l1, l2)


def test_streams_graphs_and_shared_prefix_pages():
    """Two sequences that share their prefix pages (a fork), on a side stream and captured; new lengths, trees
    and inputs in place are what a replay sees."""
    c = Case([200, 200], 6, seed=9, N=256)
    c.table[1] = c.table[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b0 = c.select(stream=s)
    o0, l0 = c.attend(b0, want_lse=True, stream=s)
    s.synchronize()
    c.check_attention(b0, o0, l0)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        b1, m1 = c.select(want_margin=True)
        o1, l1 = c.attend(b1, want_lse=True)
    gr.replay()
    assert torch.equal(b0, b1) and torch.equal(o0, o1)
    c.lens -= 45
    c.parents.copy_(_parents("chain", 2, 6, None))
    c.q.neg_()
    gr.replay()
    c.check_selection(b1, m1)
    c.check_attention(b1, o1, l1)


def test_speculative_step_end_to_end():
    """Rotate, select, attend, accept and append, then draft again: the second step's nodes match the oracle on
    a cache grown by the accepted path."""
    c = Case([150, 64, 31], 5, seed=10, N=224, kind="chain")
    f, amp = msa.msa_rope_inv_freq(64, device=DEV)
    depth = torch.arange(5, device=DEV, dtype=I32)
    pos = (c.lens[:, None] + depth).contiguous()
    q, k = msa.msa_rope_fwd([c.q, c.k], [(f, amp)] * 2, pos)
    for x, y in ((c.q, q), (c.k, k)):
        want = otree.rope(x.flatten(0, 1), f, amp, pos.flatten().cpu(), False).reshape(x.shape)
        assert (np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 5e-6).all()
    c.q, c.k = q, k
    _run(c)
    # accept nodes 0, 1, 2 of the first, none of the second, all of the third
    n_new = torch.tensor([3, 0, 5], dtype=I32, device=DEV)
    rows = torch.arange(5, device=DEV, dtype=I32).repeat(3, 1)
    msa.msa_cache_append(c.dm, c.pages, c.k, c.v, c.k_idx, c.kp, c.vp, c.kip, n_new, rows=rows)
    c.lens += n_new
    g = torch.Generator(device=DEV).manual_seed(77)
    c.q, c.k, c.v = _bf(g, *c.q.shape), _bf(g, *c.k.shape), _bf(g, *c.v.shape)
    c.q_idx, c.k_idx = _grid(g, *c.q_idx.shape), _grid(g, *c.k_idx.shape)
    _run(c)


def test_many_sequences_some_without_a_cache_or_nodes():
    """More sequences than SMs: the ragged work list, ancestor sets by several sequences per CTA."""
    g = torch.Generator().manual_seed(3)
    B = 317
    lens = torch.randint(0, 90, (B,), generator=g).tolist()
    nn = torch.randint(0, 4, (B,), generator=g).tolist()
    c = Case(lens, 3, H_q=4, H_kv=2, d=64, di=32, bk=32, topk=2, n_nodes=nn, seed=21)
    _run(c)


@pytest.mark.parametrize("nodes", ["all", "ragged", "few", "one"])
def test_more_rows_than_the_device_runs_at_once(nodes):
    """Up to 400 tiles of 128 rows (8 nodes each): full waves of CTAs, a split last wave, sequences without a node,
    tiles without a node."""
    g = torch.Generator().manual_seed(8)
    B, T = 67, 20
    nn = {"all": [T] * B, "ragged": torch.randint(0, T + 1, (B,), generator=g).tolist(), "one": [0] * (B - 1) + [T],
          "few": [20 if b % 9 == 4 else b % 2 for b in range(B)]}[nodes]
    lens = torch.randint(0, 400, (B,), generator=g).tolist()
    c = Case(lens, T, H_q=32, H_kv=2, d=64, di=32, bk=32, topk=4, n_nodes=nn, seed=22)
    blocks = c.select()
    out, lse = c.attend(blocks, want_lse=True)
    c.check_attention(blocks, out, lse, nodes=[0, 7, 8, 19])
    out2, lse2 = c.attend(blocks, want_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    b16, _ = c.attend(blocks, out_dtype=torch.bfloat16, want_lse=True)
    assert torch.equal(b16, out.to(torch.bfloat16))
    dead = torch.arange(T, device=DEV)[None] >= c.n_nodes[:, None]
    assert (out[dead] == 0).all() and torch.isneginf(lse[dead]).all()


@pytest.mark.parametrize("bk,L", [(32, 262144), (128, 262143), (64, 140001)])
def test_largest_block_counts(bk, L):
    """Up to the 8192 blocks of a sequence: every Top-k variant, lists spread over the whole page table."""
    c = Case([L - 5, L // 2], 2, H_q=16, H_kv=2, d=64, di=32, bk=bk, topk=16, seed=bk, N=L)
    _run(c)


def test_nan_and_infinite_values_stay_with_the_rows_that_see_them():
    """A NaN query, a NaN and an infinite key in a page that one node selects, a NaN key of a drafted token: only the
    rows that see them are NaN, the others as without."""
    c = Case([9 * 32 + 4], 4, H_q=8, H_kv=2, d=64, di=32, bk=32, topk=4, kind="roots", seed=31)
    lists = torch.full((1, 4, 2, 5), -1, dtype=I32, device=DEV)
    for n in range(4):
        lists[0, n, :, :4] = torch.tensor([0, 1, 2 + n, 9], device=DEV)  # block 2 + n is node n's alone
    good, glse = c.attend(lists, want_lse=True)
    c.check_attention(lists, good, glse)
    c.q[0, 0, 3] = NAN
    c.kp[int(c.table[0, 3]), 5, 1] = NAN           # block 3, group 1: node 1
    c.kp[int(c.table[0, 4]), 31, 0, 7] = float("inf")  # block 4, group 0: node 2
    c.k[0, 3, 0] = NAN                             # node 3's own key, group 0
    out, lse = c.attend(lists, want_lse=True)
    bad = torch.zeros(4, 8, dtype=torch.bool, device=DEV)
    bad[0, 3] = True
    bad[1, 4:], bad[2, :4], bad[3, :4] = True, True, True
    # (q . k with one infinite element is +-inf by the sign of q's: -inf is a weight of zero, not a NaN)
    minus = c.q[0, 2, :4, 7] < 0
    nan = torch.isnan(out[0]).all(-1) & torch.isnan(lse[0])
    assert torch.equal(nan[:2], bad[:2]) and torch.equal(nan[3], bad[3])
    assert torch.equal(nan[2, 4:], bad[2, 4:]) and torch.equal(nan[2, :4], ~minus)
    assert torch.equal(out[0][~bad], good[0][~bad]) and torch.equal(lse[0][~bad], glse[0][~bad])
    assert torch.isfinite(out[0, 2, :4][minus]).all()


def test_two_calls_at_once_on_two_streams():
    a = Case([700, 300], 8, H_q=64, H_kv=4, d=128, di=64, bk=128, topk=4, seed=41)
    b = Case([90, 1000, 5], 5, H_q=8, H_kv=2, d=64, di=32, bk=32, topk=3, seed=42)
    want = []
    for c in (a, b):
        blocks = c.select()
        want.append((blocks, c.attend(blocks)[0]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = []
        for c, s in zip((a, b), streams):
            blocks = c.select(stream=s)
            got.append((blocks, c.attend(blocks, stream=s)[0]))
        torch.cuda.synchronize()
        for (x, y), (u, v) in zip(got, want):
            assert torch.equal(x, u) and torch.equal(y, v)


def test_callers_workspace_and_output():
    c = Case([300, 40], 3, seed=51)
    ws = msa.tree_workspace(msa.MSA_OP_TREE_ATTN, c.dm, 3, DEV)
    blocks = c.select()
    out = torch.full((2, 3, 8, 64), 7.0, device=DEV)
    o, lse = c.attend(blocks, out=out, ws=ws)
    assert o is out and lse is None and torch.equal(out, c.attend(blocks)[0])
    with pytest.raises(msa.MsaError) as e:
        c.attend(blocks, ws=torch.empty(128, dtype=torch.uint8, device=DEV))
    assert e.value.code == msa.MSA_ERR_WORKSPACE
    with pytest.raises(ValueError, match="out: expected"):
        c.attend(blocks, out=out, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="parents"):
        msa.msa_tree_index_topk(c.dm, c.pages, msa.MsaTree(c.parents[:1], c.n_nodes), c.q_idx, c.k_idx, c.kip)


def test_thousands_of_sequences_with_few_nodes():
    """More sequences than a warp counts in one go: items found among 1100 sequences, most of them without a node."""
    B, T = 1100, 9
    nn = [T if b % 7 == 3 else 1 if b % 50 == 0 else 0 for b in range(B)]
    c = Case([(b * 13) % 40 for b in range(B)], T, H_q=32, H_kv=1, d=64, di=32, bk=32, topk=1, n_nodes=nn, seed=23)
    blocks = c.select()
    out, lse = c.attend(blocks, want_lse=True)
    c.check_attention(blocks, out, lse, nodes=[0, 8])


def test_a_graph_replayed_with_other_trees():
    """How the attention's work is spread depends on n_nodes on the device: a captured call follows it."""
    g = torch.Generator().manual_seed(9)
    B, T = 67, 20
    lens = torch.randint(0, 400, (B,), generator=g).tolist()
    c = Case(lens, T, H_q=32, H_kv=2, d=64, di=32, bk=32, topk=4, seed=24)
    c.attend(c.select())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blocks = c.select()
        out, lse = c.attend(blocks, want_lse=True)
    for nn in ([T] * B, [3] * B, [0] * B, [0] * (B - 1) + [T], torch.randint(0, T + 1, (B,), generator=g).tolist()):
        c.n_nodes.copy_(torch.tensor(nn, dtype=I32))
        graph.replay()
        blocks2 = c.select()
        out2, lse2 = c.attend(blocks2, want_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(blocks, blocks2) and torch.equal(out, out2) and torch.equal(lse, lse2)
    c.check_attention(blocks, out, lse, nodes=[0, 19])
