"""Host logic of rotary positions, paged caches and drafted-token trees that needs no GPU: argument checks of
the C entries and the binding, workspace sizes, inverse frequencies."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_idx_b200 as msa

P = ctypes.c_void_p


def dims(**kw):
    d = dict(B=2, N=512, H_q=4, H_kv=2, d=64, d_idx=32, block_k=32, topk=4)
    d.update(kw)
    return msa.MsaDims(**d)


def _rope(n=1, tokens=4, x_type=0, y_type=0, pos=0x7000, fn="msa_rope_fwd", **kw):
    """Status of a rope call on made-up pointers: every call here is refused before any launch."""
    segs = (msa._RopeSeg * max(n, 1))()
    for i in range(n):
        s = dict(x=0x100000 * (2 * i + 1), y=0x100000 * (2 * i + 2), x_stride=256, y_stride=256, inv_freq=0x5000, heads=4,
                 dim=64, rot=64, amp=1.0)
        s.update(kw)
        segs[i] = msa._RopeSeg(**s)
    return getattr(msa.lib(), fn)(segs if n else None, n, tokens, P(pos), 0, x_type, y_type, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), msa.MSA_ERR_INVALID_ARG), (dict(n=9, x=0x100000, y=0x900000), msa.MSA_ERR_UNSUPPORTED),
    (dict(tokens=-1), msa.MSA_ERR_INVALID_ARG), (dict(tokens=1 << 31), msa.MSA_ERR_UNSUPPORTED),
    (dict(x_type=2), msa.MSA_ERR_INVALID_ARG), (dict(y_type=-1), msa.MSA_ERR_INVALID_ARG),
    (dict(pos=0x7002), msa.MSA_ERR_INVALID_ARG), (dict(x=0), msa.MSA_ERR_INVALID_ARG),
    (dict(y=0x100008), msa.MSA_ERR_INVALID_ARG), (dict(inv_freq=0x5004), msa.MSA_ERR_INVALID_ARG),
    (dict(rot=0), msa.MSA_ERR_INVALID_ARG), (dict(rot=33), msa.MSA_ERR_INVALID_ARG),
    (dict(rot=66), msa.MSA_ERR_INVALID_ARG), (dict(amp=math.inf), msa.MSA_ERR_INVALID_ARG),
    (dict(dim=96, x_stride=384, y_stride=384), msa.MSA_ERR_UNSUPPORTED), (dict(heads=0), msa.MSA_ERR_INVALID_ARG),
    (dict(x_stride=255), msa.MSA_ERR_INVALID_ARG), (dict(x_stride=260), msa.MSA_ERR_INVALID_ARG),
    (dict(y_stride=128), msa.MSA_ERR_INVALID_ARG),
    # outputs that overlap inputs or each other
    (dict(y=0x100010), msa.MSA_ERR_INVALID_ARG), (dict(y=0x100000, y_type=1), msa.MSA_ERR_INVALID_ARG),
    (dict(y=0x100000, y_stride=512), msa.MSA_ERR_INVALID_ARG), (dict(n=2, y=0x900000), msa.MSA_ERR_INVALID_ARG),
    (dict(n=2, x=0x100000, y=0x100000), msa.MSA_ERR_INVALID_ARG),
])
@pytest.mark.parametrize("fn", ["msa_rope_fwd", "msa_rope_bwd"])
def test_rope_refusals(fn, kw, code):
    assert _rope(fn=fn, **kw) == code


def test_rope_of_no_tokens_is_accepted_without_a_launch():
    assert _rope(tokens=0) == msa.MSA_OK
    # column slices of one buffer (equal strides, disjoint columns) do not overlap
    segs = (msa._RopeSeg * 2)(msa._RopeSeg(0x100000, 0x100000, 768, 768, 0x5000, 8, 64, 64, 1.0),
                              msa._RopeSeg(0x100000 + 1024, 0x100000 + 1024, 768, 768, 0x5000, 4, 64, 64, 1.0))
    assert msa.lib().msa_rope_fwd(segs, 2, 0, None, 0, 0, 0, None) == msa.MSA_OK


def _pages(num_pages=40, table=0x1000, lens=0x2000):
    return msa._Pages(table, lens, num_pages)


def _append(d=None, pg=None, T=4, T_new=4, n_new=0x9000, rows=0, k=0x10000, ws=0, ws_bytes=0):
    d, pg = d or dims(), pg or _pages()
    return msa.lib().msa_cache_append(ctypes.byref(d.c()), ctypes.byref(pg), T, P(k), P(0x20000), P(0x30000), T_new,
                                      P(n_new), P(rows), P(0x40000), P(0x50000), P(0x60000), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=dims(H_q=5)), msa.MSA_ERR_INVALID_ARG), (dict(d=dims(block_k=16)), msa.MSA_ERR_UNSUPPORTED),
    (dict(pg=_pages(0)), msa.MSA_ERR_INVALID_ARG), (dict(pg=_pages(1 << 26)), msa.MSA_ERR_UNSUPPORTED),
    (dict(pg=_pages(table=0)), msa.MSA_ERR_INVALID_ARG), (dict(pg=_pages(lens=0x2002)), msa.MSA_ERR_INVALID_ARG),
    (dict(T=0), msa.MSA_ERR_INVALID_ARG), (dict(T_new=0), msa.MSA_ERR_INVALID_ARG), (dict(T_new=5), msa.MSA_ERR_INVALID_ARG),
    (dict(n_new=0), msa.MSA_ERR_INVALID_ARG), (dict(k=0x10002), msa.MSA_ERR_INVALID_ARG),
    (dict(rows=0x9002), msa.MSA_ERR_INVALID_ARG), (dict(ws=0x10010, ws_bytes=4096), msa.MSA_ERR_WORKSPACE),
    (dict(ws=0x10000, ws_bytes=128), msa.MSA_ERR_WORKSPACE),
])
def test_append_refusals(kw, code):
    assert _append(**kw) == code


def _copy(d=None, num_pages=8, n=2, src=0x1000, dst=0x2000, k=0x10000, ws=0, ws_bytes=0):
    return msa.lib().msa_cache_copy_pages(ctypes.byref((d or dims()).c()), num_pages, n, P(src), P(dst), P(k), P(0x20000),
                                          P(0x30000), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_pages=0), msa.MSA_ERR_INVALID_ARG), (dict(n=-1), msa.MSA_ERR_INVALID_ARG),
    (dict(n=(1 << 22) + 1), msa.MSA_ERR_UNSUPPORTED), (dict(src=0), msa.MSA_ERR_INVALID_ARG),
    (dict(dst=0x2002), msa.MSA_ERR_INVALID_ARG), (dict(k=0), msa.MSA_ERR_INVALID_ARG),
    (dict(d=dims(d=96)), msa.MSA_ERR_UNSUPPORTED), (dict(ws=0x10000, ws_bytes=8), msa.MSA_ERR_WORKSPACE),
])
def test_copy_refusals(kw, code):
    assert _copy(**kw) == code


def test_copy_of_no_pages_is_accepted_without_a_launch():
    assert _copy(n=0, src=0, dst=0) == msa.MSA_OK


def _tree(op, d=None, pg=None, T=4, parents=0x3000, n_nodes=0x4000, q=0x10000, ws=0x100000, ws_bytes=1 << 40):
    d, pg, tr = d or dims(), pg or _pages(), msa._Tree(parents, n_nodes, T)
    head = [ctypes.byref(d.c()), ctypes.byref(pg), ctypes.byref(tr), P(q), P(0x20000), P(0x30000)]
    if op == "msa_tree_index_topk":
        return msa.lib().msa_tree_index_topk(*head, P(0x40000), None, P(ws), ws_bytes, None)
    return getattr(msa.lib(), op)(*head, P(0x40000), P(0x50000), P(0x60000), P(0x70000), None, P(ws), ws_bytes, None)


@pytest.mark.parametrize("op", ["msa_tree_index_topk", "msa_tree_sparse_attn", "msa_tree_sparse_attn_bf16"])
@pytest.mark.parametrize("kw,code", [
    (dict(T=0), msa.MSA_ERR_INVALID_ARG), (dict(T=65), msa.MSA_ERR_UNSUPPORTED),
    (dict(d=dims(N=8192 * 32 + 1)), msa.MSA_ERR_UNSUPPORTED), (dict(d=dims(N=1 << 24, block_k=128)), msa.MSA_ERR_UNSUPPORTED),
    (dict(d=dims(topk=17)), msa.MSA_ERR_UNSUPPORTED), (dict(d=dims(N=0)), msa.MSA_ERR_INVALID_ARG),
    (dict(parents=0), msa.MSA_ERR_INVALID_ARG), (dict(n_nodes=0x4001), msa.MSA_ERR_INVALID_ARG),
    (dict(pg=_pages(num_pages=0)), msa.MSA_ERR_INVALID_ARG), (dict(q=0x10008), msa.MSA_ERR_INVALID_ARG),
    (dict(ws=0), msa.MSA_ERR_WORKSPACE), (dict(ws=0x100010), msa.MSA_ERR_WORKSPACE), (dict(ws_bytes=255), msa.MSA_ERR_WORKSPACE),
])
def test_tree_refusals(op, kw, code):
    assert _tree(op, **kw) == code


def test_tree_workspace_sizes():
    d = dims(B=16, N=262144, H_q=64, H_kv=4, d=128, d_idx=64, block_k=128, topk=16)
    # block maxima of every (node, group) row dominate the selection's
    n = msa.msa_tree_workspace_size(msa.MSA_OP_TREE_INDEX_TOPK, d, 16)
    assert 16 * 16 * 4 * 2048 * 4 <= n < 1.1 * 16 * 16 * 4 * 2048 * 4
    # partial outputs of at most two CTAs an SM, whatever the batch
    big = dims(B=64, N=262144, H_q=64, H_kv=4, d=128, d_idx=64, block_k=128, topk=16)
    assert msa.msa_tree_workspace_size(msa.MSA_OP_TREE_ATTN, d, 64) == msa.msa_tree_workspace_size(msa.MSA_OP_TREE_ATTN, big, 64)
    assert msa.msa_tree_workspace_size(msa.MSA_OP_TREE_ATTN, dims(B=1), 1) > 256
    for op, T in ((msa.MSA_OP_DECODE, 4), (msa.MSA_OP_TREE_ATTN, 0)):
        with pytest.raises(msa.MsaError):
            msa.msa_tree_workspace_size(op, d, T)


def test_bindings_reject_host_tensors_and_wrong_shapes():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    d = dims()
    f, amp = msa.msa_rope_inv_freq(64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        msa.msa_rope_fwd([bf(4, 2, 64)], [(f, amp)])
    with pytest.raises(ValueError, match="per tensor"):
        msa.msa_rope_bwd([bf(4, 2, 64)], [])
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        msa.msa_rope_fwd([torch.zeros(4, 2, 64, dtype=torch.float16)], [(f, amp)])
    pg, tr = msa.MsaPages(i32(2, 16), i32(2)), msa.MsaTree(i32(2, 4), i32(2))
    pools = bf(40, 32, 2, 64), bf(40, 32, 2, 64), bf(40, 32, 32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        msa.msa_cache_append(d, pg, bf(2, 4, 2, 64), bf(2, 4, 2, 64), bf(2, 4, 32), *pools, i32(2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        msa.msa_cache_copy_pages(d, [0], [1], *pools)
    with pytest.raises(ValueError, match="CUDA tensor"):
        msa.msa_tree_index_topk(d, pg, tr, bf(2, 4, 2, 32), bf(2, 4, 32), pools[2])
    with pytest.raises(ValueError, match="CUDA tensor"):
        msa.msa_tree_sparse_attn(d, pg, tr, bf(2, 4, 4, 64), bf(2, 4, 2, 64), bf(2, 4, 2, 64), *pools[:2], i32(2, 4, 2, 5))


def test_token_rows_of_views():
    x = torch.zeros(3, 5, 12, 64)
    assert msa._token_rows(x, "x") == (15, 12, 64, 768)
    assert msa._token_rows(x[:, :, 2:6], "x") == (15, 4, 64, 768)
    for bad in (x[..., ::2], x.transpose(2, 3), x[:, 1:4], x[:, :, ::2], torch.zeros(4, 64)):
        with pytest.raises(ValueError):
            msa._token_rows(bad, "x")
    assert msa._token_rows(x[:, :1, :4], "x") == (3, 4, 64, 5 * 768)


def test_inverse_frequencies():
    f, amp = msa.msa_rope_inv_freq(128)
    assert f.dtype == torch.float64 and f.numel() == 64 and amp == 1.0 and f[0] == 1.0
    assert math.isclose(float(f[-1]), 10000.0 ** (-126 / 128), rel_tol=1e-14)
    lin, _ = msa.msa_rope_inv_freq(128, scaling="linear", factor=8.0)
    assert torch.equal(lin, f / 8)
    ntk, _ = msa.msa_rope_inv_freq(128, scaling="ntk", factor=8.0)
    assert ntk[0] == 1.0 and math.isclose(float(ntk[-1]), float(f[-1]) / 8, rel_tol=1e-12)
    y, a = msa.msa_rope_inv_freq(128, scaling="yarn", factor=8.0, orig_len=4096)
    turns = f * 4096 / (2 * math.pi)
    assert math.isclose(a, 0.1 * math.log(8) + 1)
    assert torch.equal(y[turns > 40], f[turns > 40]) and torch.allclose(y[turns < 0.5], f[turns < 0.5] / 8, rtol=1e-14)
    assert ((y <= f) & (y >= f / 8 * (1 - 1e-12))).all()
    for bad in (dict(rot=3), dict(rot=0), dict(rot=4, base=1.0), dict(rot=4, scaling="other"), dict(rot=4, scaling="yarn"),
                dict(rot=4, factor=0.5)):
        with pytest.raises(ValueError):
            msa.msa_rope_inv_freq(**bad)
