"""Paged caches: appended tokens and copied pages against direct indexing (bytes are moved, so all comparisons
are exact), and what out-of-range entries leave untouched."""
import pytest
import torch

import block_sparse_attention_idx_b200 as msa

pytestmark = pytest.mark.gpu

DEV = "cuda"
I32 = torch.int32


def _bf(g, *s):
    return torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)


def _case(B, cols, T, H_kv, d, di, bk, seed, spare=2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    pages = B * cols + spare
    dm = msa.MsaDims(B, cols * bk, H_kv, H_kv, d, di, bk, 4)
    table = torch.randperm(pages, generator=g, device=DEV)[:B * cols].view(B, cols).to(I32)
    pools = [_bf(g, pages, bk, H_kv, d), _bf(g, pages, bk, H_kv, d), _bf(g, pages, bk, di)]
    new = [_bf(g, B, T, H_kv, d), _bf(g, B, T, H_kv, d), _bf(g, B, T, di)]
    return dm, g, table, pools, new


def _want(pools, new, table, lens, n_new, rows, bk):
    out = [p.clone() for p in pools]
    for b in range(table.shape[0]):
        for i in range(int(n_new[b])):
            slot = int(lens[b]) + i
            page, at, row = int(table[b, slot // bk]), slot % bk, i if rows is None else int(rows[b, i])
            for o, x in zip(out, new):
                o[page, at] = x[b, row]
    return out


@pytest.mark.parametrize("B,cols,T,H_kv,d,di,bk", [
    (1, 1, 1, 1, 64, 32, 32), (3, 4, 7, 2, 64, 32, 32), (5, 3, 64, 4, 128, 64, 64), (2, 2, 129, 8, 128, 64, 128),
    (17, 3, 33, 1, 128, 32, 64), (4, 2, 3, 4, 64, 64, 128),
])
def test_append_writes_the_slots_and_nothing_else(B, cols, T, H_kv, d, di, bk):
    dm, g, table, pools, new = _case(B, cols, T, H_kv, d, di, bk, seed=T)
    room = cols * bk - T
    lens = torch.randint(0, room + 1, (B,), generator=g, device=DEV, dtype=I32)
    lens[0] = room
    n_new = torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=I32)
    n_new[0] = T
    want = _want(pools, new, table, lens, n_new, None, bk)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    msa.msa_cache_append(dm, msa.MsaPages(table, lens), *new, *pools, n_new, ws=ws)
    assert msa.msa_get_device_status(ws) == msa.MSA_OK
    for a, b in zip(pools, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,T_new", [(16, 16), (5, 3), (4, 9), (1, 1)])
def test_append_accepted_rows(T, T_new):
    B, cols, bk = 6, 2, 32
    dm, g, table, pools, new = _case(B, cols, T, 2, 64, 32, bk, seed=50 + T)
    lens = torch.randint(0, cols * bk - T_new + 1, (B,), generator=g, device=DEV, dtype=I32)
    n_new = torch.randint(0, T_new + 1, (B,), generator=g, device=DEV, dtype=I32)
    rows = torch.randint(0, T, (B, T_new), generator=g, device=DEV, dtype=I32)  # repeats and any order too
    for b in range(B):  # unused entries may hold anything
        rows[b, int(n_new[b]):] = 12345
    want = _want(pools, new, table, lens, n_new, rows, bk)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    msa.msa_cache_append(dm, msa.MsaPages(table, lens), *new, *pools, n_new, rows=rows, ws=ws)
    assert msa.msa_get_device_status(ws) == msa.MSA_OK
    for a, b in zip(pools, want):
        assert torch.equal(a, b)


def test_append_out_of_range_entries_are_not_written_and_reported():
    B, cols, bk, T = 7, 2, 32, 4
    dm, g, table, pools, new = _case(B, cols, T, 1, 64, 32, bk, seed=3)
    N = cols * bk
    lens = torch.tensor([N - 2, -1, N, 5, 5, 5, 40], dtype=I32, device=DEV)
    n_new = torch.tensor([4, 4, 1, -3, 9, 2, 2], dtype=I32, device=DEV)
    table[5, 0] = pools[0].shape[0]  # a page past the pool
    table[3, 0] = -7                 # not read: nothing is appended there
    rows = torch.arange(T, device=DEV, dtype=I32).repeat(B, 1)
    rows[6, 1] = T                   # a row past the new tokens
    ok_n = torch.tensor([2, 0, 0, 0, 4, 0, 1], dtype=I32)
    want = _want(pools, new, table, lens.clamp(0, N), ok_n, rows, bk)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    msa.msa_cache_append(dm, msa.MsaPages(table, lens), *new, *pools, n_new, rows=rows, ws=ws)
    assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_CHECK
    for a, b in zip(pools, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("pages,n,H_kv,d,di,bk", [(2, 1, 1, 64, 32, 32), (40, 13, 4, 128, 64, 128), (9, 4, 8, 128, 32, 64),
                                                  (300, 150, 2, 64, 64, 32), (5, 0, 1, 64, 32, 32)])
def test_copy_pages(pages, n, H_kv, d, di, bk):
    g = torch.Generator(device=DEV).manual_seed(pages)
    dm = msa.MsaDims(1, bk, H_kv, H_kv, d, di, bk, 1)
    pools = [_bf(g, pages, bk, H_kv, d), _bf(g, pages, bk, H_kv, d), _bf(g, pages, bk, di)]
    order = torch.randperm(pages, generator=g, device=DEV)
    dst, src = order[:n], order[n:][torch.randint(0, pages - n, (n,), generator=g, device=DEV)]  # a source may repeat
    want = [p.clone() for p in pools]
    for w in want:
        w[dst] = w[src]
    lists = [p.clone() for p in pools]
    both = torch.cat([dst, src]).to(I32)  # slices: 4-byte alignment
    msa.msa_cache_copy_pages(dm, both[n:], both[:n], *pools)
    msa.msa_cache_copy_pages(dm, src.tolist(), dst.tolist(), *lists)
    for a, b, c in zip(pools, want, lists):
        assert torch.equal(a, b) and torch.equal(c, b)


def test_copy_pages_out_of_range_and_self_pairs():
    g = torch.Generator(device=DEV).manual_seed(1)
    dm = msa.MsaDims(1, 32, 2, 2, 64, 32, 32, 1)
    pools = [_bf(g, 6, 32, 2, 64), _bf(g, 6, 32, 2, 64), _bf(g, 6, 32, 32)]
    want = [p.clone() for p in pools]
    for w in want:
        w[2] = w[5]
    src = torch.tensor([5, 6, 0, 3, -1], dtype=I32, device=DEV)
    dst = torch.tensor([2, 1, -1, 3, 4], dtype=I32, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    msa.msa_cache_copy_pages(dm, src, dst, *pools, ws=ws)
    assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_CHECK
    for a, b in zip(pools, want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: its last pages are copied, appended to and read at the right place."""
    bk, H_kv, d, di = 128, 8, 128, 32
    pages = (1 << 32) // (bk * H_kv * d * 2) + 3  # K pool just over 4 GiB
    dm = msa.MsaDims(1, 2 * bk, H_kv, H_kv, d, di, bk, 1)
    g = torch.Generator(device=DEV).manual_seed(2)
    pools = [torch.zeros(pages, bk, H_kv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pools.append(torch.zeros(pages, bk, di, dtype=torch.bfloat16, device=DEV))
    table = torch.tensor([[0, pages - 1]], dtype=I32, device=DEV)
    new = [_bf(g, 1, 3, H_kv, d), _bf(g, 1, 3, H_kv, d), _bf(g, 1, 3, di)]
    lens = torch.tensor([bk + 5], dtype=I32, device=DEV)
    msa.msa_cache_append(dm, msa.MsaPages(table, lens), *new, *pools, torch.tensor([3], dtype=I32, device=DEV))
    msa.msa_cache_copy_pages(dm, [pages - 1], [pages - 2], *pools)
    for p, x in zip(pools, new):
        assert torch.equal(p[-1, 5:8], x[0]) and torch.equal(p[-2], p[-1])
        assert not p[-1, :5].any() and not p[-1, 8:].any() and not p[:-2].any()


def test_streams_and_graphs():
    B, cols, bk, T = 2, 2, 32, 4
    dm, g, table, pools, new = _case(B, cols, T, 2, 64, 32, bk, seed=4)
    lens = torch.tensor([3, 30], dtype=I32, device=DEV)
    n_new = torch.tensor([4, 4], dtype=I32, device=DEV)
    want = _want(_want(pools, new, table, lens, n_new, None, bk), new, table, lens + 4, n_new, None, bk)
    pg = msa.MsaPages(table, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    msa.msa_cache_append(dm, pg, *new, *pools, n_new, stream=s)
    s.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        msa.msa_cache_append(dm, pg, *new, *pools, n_new)
    lens += 4
    gr.replay()
    for a, b in zip(pools, want):
        assert torch.equal(a, b)


def test_paged_cache_forks_and_compaction_on_the_device():
    """PagedCache end to end: a prompt, two forks that diverge, one freed, the pool compacted; every sequence's
    tokens stay what was appended."""
    from block_sparse_attention_idx_b200.pages import PagedCache

    g = torch.Generator(device=DEV).manual_seed(12)
    dm = msa.MsaDims(1, 400, 8, 2, 64, 32, 32, 4)
    c = PagedCache(dm, 40)
    want = {}

    def grow(seqs, T, rows=None):
        x = [_bf(g, len(seqs), T, 2, 64), _bf(g, len(seqs), T, 2, 64), _bf(g, len(seqs), T, 32)]
        c.append(seqs, *x, rows=rows)
        for i, s in enumerate(seqs):
            pick = list(range(T)) if rows is None else rows[i]
            want[s] = [torch.cat([w, t[i, pick]]) for w, t in zip(want[s], x)]

    def check():
        for s, w in want.items():
            pages = torch.tensor(c.page_list(s), device=DEV)
            for pool, t in zip((c.k_pool, c.v_pool, c.k_idx_pool), w):
                assert torch.equal(pool[pages].flatten(0, 1)[:c.length(s)], t)

    a, z = c.new(), c.new()
    for s in (a, z):
        want[s] = [_bf(g, 0, 2, 64), _bf(g, 0, 2, 64), _bf(g, 0, 32)]
    grow([z, a], 75)
    b = c.fork(a)
    want[b] = list(want[a])
    grow([a, b], 7, rows=[[0, 2, 6], [1, 2, 3, 4]])
    check()
    c.free(z)
    del want[z]
    used = c.compact()
    assert max(c.page_list(a) + c.page_list(b)) < used == 4
    check()
    grow([b, a], 33)
    check()


def test_paged_cache_on_another_stream():
    """The index tensors of an append on a side stream stay intact while it waits there, whatever the current stream
    allocates and writes meanwhile."""
    from block_sparse_attention_idx_b200.pages import PagedCache

    c = PagedCache(msa.MsaDims(1, 256, 2, 2, 64, 32, 32, 2), 16)
    for p in (c.k_pool, c.v_pool, c.k_idx_pool):
        p.zero_()
    g = torch.Generator(device=DEV).manual_seed(5)
    k, v, ki = _bf(g, 2, 9, 2, 64), _bf(g, 2, 9, 2, 64), _bf(g, 2, 9, 32)
    side, here, seqs, rows = torch.cuda.Stream(), torch.cuda.Stream(), [c.new(), c.new()], [[0, 3, 8], [1, 2]]
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        c.append([c.new(), c.new()], k, v, ki, rows=rows)  # (the kernels are loaded)
        torch.zeros(4, dtype=I32, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        c.append(seqs, k, v, ki, rows=rows, stream=side)
        held = [torch.zeros(4, dtype=I32, device=DEV) for _ in range(16)]  # may take what is free for reuse here
    torch.cuda.synchronize()
    assert len(held) == 16
    for b, s in enumerate(seqs):
        page = c.page_list(s)[0]
        assert torch.equal(c.k_pool[page, :len(rows[b])], k[b, rows[b]])
        assert torch.equal(c.v_pool[page, :len(rows[b])], v[b, rows[b]])
        assert torch.equal(c.k_idx_pool[page, :len(rows[b])], ki[b, rows[b]])
