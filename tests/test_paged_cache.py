"""Page bookkeeping (PagedCache) on the CPU: the two device operations are replaced by plain CPU copies, and random
sequences of operations are checked against a model that keeps each sequence's tokens as a list."""
import random

import pytest
import torch

import block_sparse_attention_idx_b200 as msa
from block_sparse_attention_idx_b200.pages import PagedCache


def _fake_copy(dims, src, dst, k, v, ki, ws=None, stream=None):
    assert len(src) == len(dst) == len(set(dst)) and not set(src) & set(dst)
    for p in (k, v, ki):
        p[list(dst)] = p[list(src)]


def _fake_append(dims, pages, k, v, k_idx, kp, vp, kip, n_new, rows=None, ws=None, stream=None):
    bk = dims.block_k
    written = set()
    for b in range(dims.B):
        for i in range(int(n_new[b])):
            slot = int(pages.cache_len[b]) + i
            at = int(pages.page_table[b, slot // bk]), slot % bk
            assert at not in written  # no two tokens share a slot
            written.add(at)
            row = i if rows is None else int(rows[b, i])
            kp[at], vp[at], kip[at] = k[b, row], v[b, row], k_idx[b, row]


@pytest.fixture
def cache(monkeypatch):
    monkeypatch.setattr(msa, "msa_cache_copy_pages", _fake_copy)
    monkeypatch.setattr(msa, "msa_cache_append", _fake_append)

    def make(num_pages=12, N=200, bk=32):
        return PagedCache(msa.MsaDims(1, N, 1, 1, 64, 32, bk, 2), num_pages, device="cpu")

    return make


def _tokens(B, T, tag):
    """New tokens whose first element tells which one it is."""
    k = torch.zeros(B, T, 1, 64, dtype=torch.bfloat16)
    k[:, :, 0, 0] = torch.tensor(tag, dtype=torch.bfloat16)
    return k, k + 1, k[:, :, 0, :32] + 2


def _read(c, s):
    bk = c.dims.block_k
    pages = c.page_list(s)
    out = [float(c.k_pool[pages[p // bk], p % bk, 0, 0]) for p in range(c.length(s))]
    assert out == [float(c.v_pool[pages[p // bk], p % bk, 0, 0]) - 1 for p in range(c.length(s))]
    assert out == [float(c.k_idx_pool[pages[p // bk], p % bk, 0]) - 2 for p in range(c.length(s))]
    return out


def _consistent(c):
    held = {}
    for pages, n in c._seqs.values():
        assert len(pages) == len(set(pages)) and len(pages) >= -(-n // c.dims.block_k)
        for p in pages:
            held[p] = held.get(p, 0) + 1
    assert [held.get(p, 0) for p in range(c.num_pages)] == c._refs
    assert sorted(c._free) == [p for p in range(c.num_pages) if p not in held]


def test_append_fork_copy_on_write_and_free(cache):
    c = cache()
    a = c.new()
    c.append([a], *_tokens(1, 40, [list(range(40))]))
    b = c.fork(a)
    assert c.page_list(a) == c.page_list(b) and c.free_pages == 10
    c.append([b], *_tokens(1, 1, [[77.0]]))  # the shared, partly filled page is copied, the full one is not
    assert c.page_list(a)[0] == c.page_list(b)[0] and c.page_list(a)[1] != c.page_list(b)[1]
    c.append([a], *_tokens(1, 1, [[88.0]]))  # now its own: no copy
    assert c.free_pages == 9
    assert _read(c, a) == list(range(40)) + [88.0] and _read(c, b) == list(range(40)) + [77.0]
    c.free(a)
    assert _read(c, b) == list(range(40)) + [77.0] and c.free_pages == 10
    c.free(b)
    assert c.free_pages == 12
    _consistent(c)


def test_full_last_page_is_shared_without_a_copy(cache):
    c = cache()
    a = c.new()
    c.append([a], *_tokens(1, 32, [list(range(32))]))
    b = c.fork(a)
    c.append([a, b], *_tokens(2, 1, [[1.0], [2.0]]))
    assert c.page_list(a)[0] == c.page_list(b)[0] and c.free_pages == 9


def test_both_owners_in_one_append_take_one_copy(cache):
    c = cache()
    a = c.new()
    c.append([a], *_tokens(1, 5, [list(range(5))]))
    b = c.fork(a)
    c.append([a, b], *_tokens(2, 2, [[6.0, 7.0], [8.0, 9.0]]))
    assert c.free_pages == 10
    assert _read(c, a)[5:] == [6.0, 7.0] and _read(c, b)[5:] == [8.0, 9.0]
    _consistent(c)


def test_reserved_pages_are_not_shared_by_a_fork(cache):
    c = cache()
    a = c.new()
    c.append([a], *_tokens(1, 5, [list(range(5))]))
    c.reserve([a], [70])
    b = c.fork(a)
    c.append([a, b], *_tokens(2, 40, [list(range(50, 90)), list(range(100, 140))]))
    assert _read(c, a)[5:] == list(range(50, 90)) and _read(c, b)[5:] == list(range(100, 140))
    _consistent(c)


def test_rows_counts_and_truncate(cache):
    c = cache()
    a, b, e = c.new(), c.new(), c.new()
    c.append([a, b, e], *_tokens(3, 4, [[0, 1, 2, 3], [10, 11, 12, 13], [20, 21, 22, 23]]), rows=[[0, 2], [], [3, 1, 0]])
    assert _read(c, a) == [0, 2] and _read(c, b) == [] and _read(c, e) == [23, 21, 20]
    c.append([b], *_tokens(1, 40, [list(range(40))]), counts=[35])
    c.truncate(b, 31)
    assert _read(c, b) == list(range(31)) and len(c.page_list(b)) == 1
    c.truncate(b, 0)
    assert c.page_list(b) == []
    _consistent(c)


def test_errors_change_nothing(cache):
    c = cache(num_pages=3, N=128)
    a = c.new()
    c.append([a], *_tokens(1, 50, [list(range(50))]))
    b = c.fork(a)
    before = (c.page_list(a), c.page_list(b), c.free_pages)
    for call in (lambda: c.append([a, b], *_tokens(2, 40, [[0.0] * 40] * 2)),  # needs 3 pages, 1 free
                 lambda: c.append([a], *_tokens(1, 79, [[0.0] * 79])),         # past the capacity
                 lambda: c.reserve([a, a], [1, 1]), lambda: c.reserve([a], [1, 2]), lambda: c.reserve([a], [-1]),
                 lambda: c.reserve([99], [1]), lambda: c.truncate(a, 51), lambda: c.free(99), lambda: c.fork(99),
                 lambda: c.append([a], *_tokens(1, 2, [[0.0, 0.0]]), rows=[[2]]),
                 lambda: c.append([a], *_tokens(1, 2, [[0.0, 0.0]]), counts=[3]),
                 lambda: c.append([a], *_tokens(1, 2, [[0.0, 0.0]]), counts=[1], rows=[[0, 1]]),
                 lambda: c.append([a, b], *_tokens(1, 2, [[0.0, 0.0]])), lambda: c.pages([]),
                 lambda: PagedCache(c.dims, 0, device="cpu")):
        with pytest.raises(ValueError):
            call()
        assert before == (c.page_list(a), c.page_list(b), c.free_pages)
        _consistent(c)


def test_a_copy_that_cannot_start_changes_nothing(cache, monkeypatch):
    c = cache()
    a, gone = c.new(), c.new()
    k, v, ki = _tokens(1, 40, [list(range(40))])
    c.append([gone], k, v, ki)
    c.append([a], k, v, ki)
    f = c.fork(a)
    c.free(gone)
    before = ([list(c._refs), list(c._free)], {s: c.page_list(s) for s in (a, f)})

    def refuse(*args, **kw):
        raise ValueError("another device's stream")

    monkeypatch.setattr(msa, "msa_cache_copy_pages", refuse)
    for call in (lambda: c.append([f], k, v, ki), lambda: c.reserve([a, f], [1, 1]), c.compact):
        with pytest.raises(ValueError, match="another device"):
            call()
        assert before == ([list(c._refs), list(c._free)], {s: c.page_list(s) for s in (a, f)})
        assert _read(c, a) == _read(c, f) == list(range(40))


def test_page_table_and_lengths(cache):
    c = cache(N=100)
    a, b = c.new(), c.new()
    c.append([a], *_tokens(1, 70, [[0.0] * 70]))
    pg = c.pages([b, a])
    assert pg.page_table.shape == (2, 4) and pg.page_table.dtype == torch.int32
    assert pg.cache_len.tolist() == [0, 70] and pg.page_table[1, :3].tolist() == c.page_list(a)
    assert c.dims_for(2).B == 2 and c.dims_for(2).N == 100


@pytest.mark.parametrize("seed", range(6))
def test_random_operations_match_the_model(cache, seed):
    r = random.Random(seed)
    c = cache(num_pages=20, N=150)
    model, tag = {}, 0
    for _ in range(250):
        op = r.choice(["new", "append", "append", "append", "reserve", "fork", "free", "truncate", "compact"])
        if op == "new" and len(model) < 6:
            model[c.new()] = []
        elif op == "append" and model:
            seqs = r.sample(sorted(model), r.randint(1, len(model)))
            T = r.randint(1, 40)
            vals = [[float((tag := tag + 1) % 250) for _ in range(T)] for _ in seqs]
            rows = [sorted(r.sample(range(T), r.randint(0, T))) for _ in seqs] if r.random() < 0.5 else None
            try:
                c.append(seqs, *_tokens(len(seqs), T, vals), rows=rows)
            except ValueError:
                _consistent(c)
                continue
            for i, s in enumerate(seqs):
                model[s] = model[s] + (vals[i] if rows is None else [vals[i][x] for x in rows[i]])
        elif op == "reserve" and model:
            seqs = r.sample(sorted(model), r.randint(1, len(model)))
            try:
                c.reserve(seqs, [r.randint(0, 70) for _ in seqs])
            except ValueError:
                pass
        elif op == "fork" and model and len(model) < 8:
            s = r.choice(sorted(model))
            model[c.fork(s)] = list(model[s])
        elif op == "free" and len(model) > 2:
            s = r.choice(sorted(model))
            c.free(s)
            del model[s]
        elif op == "truncate" and model:
            s = r.choice(sorted(model))
            n = r.randint(0, len(model[s]))
            c.truncate(s, n)
            model[s] = model[s][:n]
        elif op == "compact":
            used = c.compact()
            assert all(p < used for s in model for p in c.page_list(s)) and used == c.num_pages - c.free_pages
        _consistent(c)
        for s, want in model.items():
            assert _read(c, s) == want
