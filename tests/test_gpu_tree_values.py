"""Infinities, NaN and the largest values in the tree attention: they belong to the rows that see their token, in their
column, and to no others, although the nodes of a tree share the products over their blocks.

Finite outputs are held to the bound of test_gpu_tree_weights.py, 2 (2^-8 / (1 - 2^-8) + 3e-5) dev + 4e-5 mag with
dev = sum_j w_j |v_j - o|, mag = sum_j w_j |v_j|, and half a step of a bf16 output."""
import numpy as np
import pytest
import torch

from test_gpu_tree import Case

pytestmark = pytest.mark.gpu

DEV = "cuda"
I32 = torch.int32
INF, NAN = float("inf"), float("nan")
LAYOUTS = [dict(H_q=8, H_kv=2, d=64, di=32, bk=32, topk=4), dict(H_q=32, H_kv=1, d=128, di=32, bk=128, topk=4),
           dict(H_q=64, H_kv=4, d=128, di=64, bk=64, topk=4)]


def _node(c, lists, b, n):
    """Output, dev and mag of a node over the tokens that it sees, in 64 bits, each column on its own."""
    K, V, _ = c.virtual(b, n)
    G = c.od.H_q // c.od.H_kv
    out, dev, mag = np.zeros((3, c.od.H_q, c.od.d))
    for h in range(c.od.H_q):
        ids = sorted({int(x) for x in lists[b, n, h // G] if x >= 0})
        J = [j for x in ids for j in range(x * c.od.block_k, min((x + 1) * c.od.block_k, K.shape[0]))]
        if not J:
            continue
        z = K[J, h // G].double().numpy() @ c.q[b, n, h].double().cpu().numpy() / c.od.d ** 0.5
        w = np.exp(z - z.max())
        w /= w.sum()
        v = V[J, h // G].double().numpy()
        with np.errstate(invalid="ignore"):
            out[h] = (w[:, None] * v).sum(0)
            dev[h] = (w[:, None] * np.abs(v - out[h])).sum(0)
            mag[h] = (w[:, None] * np.abs(v)).sum(0)
    return out, dev, mag


def _check(c, lists, got, sequences=None):
    half = torch.finfo(got.dtype).eps / 2
    g, ids = got.double().cpu().numpy(), lists.cpu().numpy()
    for b in range(c.dm.B) if sequences is None else sequences:
        for n in range(int(c.n_nodes[b])):
            o, dev, mag = _node(c, ids, b, n)
            assert np.array_equal(np.isnan(o), np.isnan(g[b, n])), (b, n)
            strange = ~np.isfinite(o)
            assert np.array_equal(o[strange], g[b, n][strange], equal_nan=True), (b, n)
            with np.errstate(invalid="ignore"):
                tol = 2 * (2.0 ** -8 / (1 - 2.0 ** -8) + 3e-5) * dev + 4e-5 * mag
                tol = tol * (1 + half) + half * np.abs(o)
                assert (np.abs(g[b, n] - o) <= tol)[~strange].all(), (b, n)
    return g


def _case(layout, B=1, T=4, seed=71, **kw):
    """Nodes over the cache, each with blocks 0, 1, its own block 2 + n and the local one."""
    bk = layout["bk"]
    c = Case([(T + 5) * bk + 4] * B, T, kind="roots", seed=seed, **layout, **kw)
    lists = torch.full((B, T, c.dm.H_kv, 5), -1, dtype=I32, device=DEV)
    for n in range(T):
        lists[:, n, :, :4] = torch.tensor([0, 1, 2 + n, T + 5], device=DEV)
    return c, lists


@pytest.mark.parametrize("layout", LAYOUTS, ids=["bk32", "bk128", "bk64"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(layout, out):
    bk = layout["bk"]
    c, lists = _case(layout)
    clean, clse = c.attend(lists, want_lse=True, out_dtype=out)
    _check(c, lists, clean)
    g = c.dm.H_kv - 1
    c.vp[int(c.table[0, 3]), 5, g, 3] = NAN        # block 3: node 1's alone
    c.vp[int(c.table[0, 3]), 6, 0, 9] = -INF
    c.vp[int(c.table[0, 4]), bk - 1, 0, 60] = INF  # block 4: node 2's alone
    c.v[0, 3, 0, 17] = NAN                         # node 3's own token, which no other node sees
    got, lse = c.attend(lists, want_lse=True, out_dtype=out)
    g2 = _check(c, lists, got)
    assert np.isnan(g2[0, 1]).any() and np.isinf(g2[0, 2]).any() and np.isnan(g2[0, 3]).any()
    assert np.isfinite(g2[0, 0]).all() and torch.equal(lse, clse)
    c.vp[int(c.table[0, 1]), 2, 0, 40] = INF       # block 1: everybody's
    c.vp[int(c.table[0, 4]), 0, 0, 40] = -INF      # and of the other sign for node 2: NaN
    _check(c, lists, c.attend(lists, out_dtype=out)[0])


def test_whole_items_and_split_ones_agree_on_what_is_finite():
    """With items enough that none is split, and with one whose keys go to several CTAs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for B in (1, sms + 1):
        c, lists = _case(LAYOUTS[0], B=B, T=3, seed=72)
        c.vp[c.table[:, 3].long(), 31] = NAN
        c.v[:, 0] = INF
        got, _ = c.attend(lists)
        finite = torch.isfinite(got).flatten(2).all(-1)
        assert torch.equal(finite, torch.tensor([False, False, True], device=DEV).expand(B, 3))
        assert torch.isposinf(got[:, 0]).all() and torch.isnan(got[:, 1]).all()
        few = [0, B - 1]
        g, ids = got.double().cpu().numpy(), lists.cpu().numpy()
        for b in few:
            o, dev, mag = _node(c, ids, b, 2)
            assert (np.abs(g[b, 2] - o) <= 2 * (2.0 ** -8 / (1 - 2.0 ** -8) + 3e-5) * dev + 4e-5 * mag).all()


@pytest.mark.parametrize("kind", ["chain", "roots"])
def test_a_drafted_value_reaches_its_descendants_alone(kind):
    c = Case([70], 6, kind=kind, seed=73, n_nodes=[5], H_q=16, H_kv=2, d=64, di=32, bk=32, topk=2)
    blocks = c.select()
    c.v[0, 2] = NAN
    got, _ = c.attend(blocks)
    bad = torch.isnan(got[0]).flatten(1).any(-1).tolist()
    assert bad == ([False, False, True, True, True, False] if kind == "chain" else [False, False, True, False, False, False])
    _check(c, blocks, got)


def test_the_largest_values_do_not_overflow():
    """V up to 2^127, and keys whose weights the lazily raised maximum leaves above 1 (in whole items): the output is a
    mean of V."""
    B = torch.cuda.get_device_properties(0).multi_processor_count + 1
    c = Case([300] * B, 3, H_q=8, H_kv=2, d=64, di=32, bk=32, topk=8, seed=74)
    for x in (c.v, c.vp):
        x.mul_(2.0 ** 124)
    for p in range(300 // 32 + 1):
        c.kp[c.table[:, p].long()] *= 1 + p / 4
    blocks = c.select()
    got, _ = c.attend(blocks)
    assert torch.isfinite(got).all()
    _check(c, blocks, got, sequences=[0, B - 1])


def test_a_bad_value_in_a_captured_call():
    c, lists = _case(LAYOUTS[1], B=2, seed=75)
    c.attend(lists)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = c.attend(lists, out_dtype=torch.bfloat16)
    graph.replay()
    clean = out.clone()
    page = c.vp[int(c.table[1, 2])]
    keep = page.clone()
    page[7] = NAN  # block 2 of the second sequence: its node 0
    graph.replay()
    assert torch.equal(out[0], clean[0]) and torch.isnan(out[1, 0]).all() and torch.isfinite(out[1, 1:]).all()
    page.copy_(keep)
    graph.replay()
    assert torch.equal(out, clean)


@pytest.mark.parametrize("layout", LAYOUTS, ids=["bk32", "bk128", "bk64"])
def test_logits_of_minus_infinity_are_weights_of_zero(layout):
    """Block 2's keys are -inf in one element: by the sign of its query a row of node 0 has logits of -inf, which count
    for nothing, or +inf, which make it NaN. With block 2 alone nothing is left: output 0 and LSE -inf, as with no token."""
    c, lists = _case(layout)
    c.kp[int(c.table[0, 2]), :, :, 7] = -INF
    out, lse = c.attend(lists, want_lse=True)
    without = lists.clone()
    without[:, 0, :, 2] = -1
    _, l2 = c.attend(without, want_lse=True)
    plus = c.q[0, 0, :, 7] < 0
    assert plus.any() and not plus.all() and not (c.q[0, 0, :, 7] == 0).any()
    assert torch.isnan(out[0, 0, plus]).all() and torch.isnan(lse[0, 0, plus]).all()
    # the others as over the lists without block 2 (their sums may be cut elsewhere: equal to the bounds, not in bits)
    ids, keep = without.cpu().numpy(), torch.ones(4, c.dm.H_q, dtype=torch.bool, device=DEV)
    keep[0] = ~plus
    for n in range(4):
        o, dev, mag = _node(c, ids, 0, n)
        tol = 2 * (2.0 ** -8 / (1 - 2.0 ** -8) + 3e-5) * dev + 4e-5 * mag
        ok = np.abs(out[0, n].double().cpu().numpy() - o) <= tol
        assert ok[keep[n].cpu().numpy()].all()
    assert (lse[0] - l2[0])[keep].abs().max() <= 6e-5
    alone = torch.full_like(lists, -1)
    alone[:, 0, :, 0] = 2
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = c.attend(alone, want_lse=True, out_dtype=dtype)
        assert (out[0, 0, ~plus] == 0).all() and torch.isneginf(lse[0, 0, ~plus]).all()
        assert torch.isnan(out[0, 0, plus]).all() and (out[0, 1:] == 0).all() and torch.isneginf(lse[0, 1:]).all()


def test_a_value_that_is_not_finite_counts_however_small_its_weight():
    """Block 0 weighs e^-1000 and holds a NaN and an infinity: by the definition's 0 times either, NaN in their columns for
    the rows that see it. In one CTA, and where the block has a CTA of its own and the merge joins them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for B in (1, sms + 1):
        c, lists = _case(LAYOUTS[1], B=B, T=2, seed=76)
        lists[:, 1, :, 0] = -1  # node 1 does not see block 0
        c.q[..., 0] = 8.0
        c.kp[c.table[:, 0].long(), :, :, 0] = -2048.0  # logits of about -1448 against others of order 10
        c.vp[c.table[:, 0].long(), 3, :, 5] = NAN
        c.vp[c.table[:, 0].long(), 4, :, 6] = INF
        out, lse = c.attend(lists, want_lse=True)
        bad = torch.isnan(out).all(0).all(1)
        assert torch.isnan(out[:, 0, :, 5:7]).all() and torch.isfinite(out[:, 1]).all() and torch.isfinite(lse).all()
        assert bad[0, 5] and bad[0, 6] and int((~torch.isfinite(out)).sum()) == 2 * B * c.dm.H_q


@pytest.mark.parametrize("layout", LAYOUTS, ids=["bk32", "bk128", "bk64"])
@pytest.mark.parametrize("B", [1, 150])
def test_the_output_in_place_of_the_queries(layout, B):
    """bf16 outputs written over q, rows that are evaluated token by token among them."""
    c, lists = _case(layout, B=B, seed=77)
    c.vp[c.table[:, 3].long(), 5, 0, 3] = NAN
    c.vp[c.table[:, 4].long(), 6, :, 9] = INF
    want, wlse = c.attend(lists, want_lse=True, out_dtype=torch.bfloat16)
    got, lse = c.attend(lists, want_lse=True, out_dtype=torch.bfloat16, out=c.q)
    assert got is c.q and torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wlse)
