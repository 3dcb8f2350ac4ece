"""Page bookkeeping of the paged K / V / K_idx caches: which pages belong to which sequence.

The pools live on the device; everything here is host state (lists of page numbers, reference counts), and the
only device work is msa_cache_append and msa_cache_copy_pages. A page holds one KV block. Sequences may share
pages: a fork shares all of its parent's, and since only a sequence's last, partly filled page is ever written, that
one is copied when one of its owners is appended to (copy on write), the others never.

Typical serving step: ``pages(seqs)`` and the tree calls, then ``append(seqs, k, v, k_idx, counts, rows)`` with the
accepted nodes. Calls on one PagedCache are ordered by the caller (one thread, one stream at a time).
"""
from __future__ import annotations

import torch

import block_sparse_attention_idx_b200 as msa


class PagedCache:
    """Pools of num_pages pages and the sequences in them. dims gives the head layout, block_k and, as N, the
    capacity of a sequence; dims.B is not used."""

    def __init__(self, dims: "msa.MsaDims", num_pages: int, device="cuda"):
        if num_pages < 1:
            raise ValueError(f"num_pages must be at least 1, got {num_pages}")
        self.dims = dims
        self.num_pages = num_pages
        self.cols = -(-dims.N // dims.block_k)
        shape = (num_pages, dims.block_k, dims.H_kv, dims.d)
        self.k_pool = torch.empty(shape, dtype=torch.bfloat16, device=device)
        self.v_pool = torch.empty(shape, dtype=torch.bfloat16, device=device)
        self.k_idx_pool = torch.empty(num_pages, dims.block_k, dims.d_idx, dtype=torch.bfloat16, device=device)
        self._free = list(range(num_pages - 1, -1, -1))  # the lowest page number is handed out next
        self._refs = [0] * num_pages
        self._seqs: dict[int, list] = {}  # handle -> [page numbers, length]
        self._next = 0

    # ------------------------------------------------------------------------------------ queries
    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        return self._get(seq)[1]

    def page_list(self, seq: int) -> list[int]:
        """The sequence's page numbers, in position order."""
        return list(self._get(seq)[0])

    def dims_for(self, batch: int) -> "msa.MsaDims":
        """The cache's dims for a call over `batch` of its sequences."""
        d = self.dims
        return msa.MsaDims(batch, d.N, d.H_q, d.H_kv, d.d, d.d_idx, d.block_k, d.topk, d.scale, d.scale_idx)

    def pages(self, seqs) -> "msa.MsaPages":
        """Page table and lengths of these sequences, on the device (a copy: later appends do not change it)."""
        rows = [self._get(s) for s in seqs]
        if not rows:
            raise ValueError("no sequences")
        dev = self.k_pool.device
        table = torch.tensor([p + [0] * (self.cols - len(p)) for p, _ in rows], dtype=torch.int32)
        lens = torch.tensor([n for _, n in rows], dtype=torch.int32)
        return msa.MsaPages(table.to(dev), lens.to(dev))

    def _get(self, seq: int) -> list:
        try:
            return self._seqs[seq]
        except KeyError:
            raise ValueError(f"no sequence {seq}") from None

    # ------------------------------------------------------------------------- sequences and pages
    def new(self) -> int:
        """An empty sequence; returns its handle."""
        return self._add([], 0)

    def fork(self, seq: int) -> int:
        """A new sequence with the same tokens, sharing every page that holds some (not those only reserved)."""
        pages, n = self._get(seq)
        pages = pages[:-(-n // self.dims.block_k)]
        for p in pages:
            self._refs[p] += 1
        return self._add(pages, n)

    def free(self, seq: int) -> None:
        """Forgets the sequence; pages that no other sequence holds are free again."""
        pages, _ = self._get(seq)
        del self._seqs[seq]
        self._release(pages)

    def truncate(self, seq: int, length: int) -> None:
        """Keeps the first `length` tokens."""
        pages, n = self._get(seq)
        if not 0 <= length <= n:
            raise ValueError(f"length must be in [0, {n}], got {length}")
        keep = -(-length // self.dims.block_k)
        self._release(pages[keep:])
        self._seqs[seq] = [pages[:keep], length]

    def _add(self, pages, n) -> int:
        handle, self._next = self._next, self._next + 1
        self._seqs[handle] = [pages, n]
        return handle

    def _release(self, pages) -> None:
        for p in pages:
            self._refs[p] -= 1
            if self._refs[p] == 0:
                self._free.append(p)

    def _take(self) -> int:
        p = self._free.pop()
        self._refs[p] = 1
        return p

    def reserve(self, seqs, counts, stream=None) -> None:
        """Pages for counts[i] more tokens of sequence seqs[i], and a copy of its last page where that is partly
        filled and shared. Raises, with nothing changed, if a sequence would pass the capacity or the pages do not
        suffice."""
        seqs, counts = list(seqs), [int(c) for c in counts]
        if len(seqs) != len(counts) or len(set(seqs)) != len(seqs):
            raise ValueError("need one count per sequence, and no sequence twice")
        bk = self.dims.block_k
        need, shared = 0, {}
        for s, c in zip(seqs, counts):
            pages, n = self._get(s)
            if c < 0 or n + c > self.dims.N:
                raise ValueError(f"sequence {s} of {n} tokens cannot grow by {c} (capacity {self.dims.N})")
            need += max(0, -(-(n + c) // bk) - len(pages))
            if c and n % bk and self._refs[pages[n // bk]] > 1:
                shared[pages[n // bk]] = shared.get(pages[n // bk], 0) + 1
        # of a page's owners that are appended to, each needs a copy, except one if nobody else holds it
        need += sum(min(k, self._refs[p] - 1) for p, k in shared.items())
        if need > len(self._free):
            raise ValueError(f"{need} pages needed, {len(self._free)} free")
        copies, owners = [], {}  # (sequence, page) to copy; owners that a shared page has left
        for s, c in zip(seqs, counts):
            pages, n = self._seqs[s]
            if c and n % bk:
                p = pages[n // bk]
                owners.setdefault(p, self._refs[p])
                if owners[p] > 1:
                    copies.append((s, p))
                    owners[p] -= 1
        if copies:  # before anything changes: the call may raise
            src, dst = [p for _, p in copies], self._free[:-len(copies) - 1:-1]
            msa.msa_cache_copy_pages(self.dims, src, dst, self.k_pool, self.v_pool, self.k_idx_pool, stream=stream)
        for s, p in copies:
            pages, n = self._seqs[s]
            pages[n // bk] = self._take()
            self._refs[p] -= 1
        for s, c in zip(seqs, counts):
            pages, n = self._seqs[s]
            while len(pages) * bk < n + c:
                pages.append(self._take())

    def append(self, seqs, k, v, k_idx, counts=None, rows=None, stream=None) -> None:
        """Writes counts[i] new tokens (default: all T) behind sequence seqs[i]: the first rows of k, v
        [B,T,H_kv,d], k_idx [B,T,d_idx], or rows[i] (lists of row numbers, e.g. an accepted path of tree nodes, whose
        lengths are then the counts). Reserves what is needed first; arguments that do not fit are refused before that."""
        seqs, d = list(seqs), self.dims
        T = k.shape[1] if k.dim() == 4 else 0
        shape = (len(seqs), T, d.H_kv, d.d)
        for t, name, want in ((k, "k", shape), (v, "v", shape), (k_idx, "k_idx", (len(seqs), T, d.d_idx))):
            if tuple(t.shape) != want or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.device != self.k_pool.device:
                raise ValueError(f"{name}: expected contiguous torch.bfloat16 {want} on {self.k_pool.device}, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
        if rows is not None:
            rows = [[int(x) for x in r] for r in rows]
            if counts is not None and [int(c) for c in counts] != [len(r) for r in rows]:
                raise ValueError("counts and the lengths of rows differ")
            if any(not 0 <= x < T for r in rows for x in r):
                raise ValueError(f"row numbers must be in [0, {T})")
            counts = [len(r) for r in rows]
        counts = [T] * len(seqs) if counts is None else [int(c) for c in counts]
        if len(counts) != len(seqs):
            raise ValueError(f"{len(seqs)} sequences, {len(counts)} counts")
        if rows is None and any(c > T for c in counts):
            raise ValueError(f"counts must be at most {T}")
        self.reserve(seqs, counts, stream=stream)
        if not any(counts):
            return
        dev = self.k_pool.device
        with msa._on(stream):  # the index tensors belong to the stream that reads them
            n_new = torch.tensor(counts, dtype=torch.int32).to(dev)
            row_t = None
            if rows is not None:
                width = max(counts)
                row_t = torch.tensor([r + [0] * (width - len(r)) for r in rows], dtype=torch.int32).to(dev)
            msa.msa_cache_append(self.dims_for(len(seqs)), self.pages(seqs), k, v, k_idx, self.k_pool, self.v_pool,
                                 self.k_idx_pool, n_new, rows=row_t, stream=stream)
        for s, c in zip(seqs, counts):
            self._seqs[s][1] += c

    def compact(self, stream=None) -> int:
        """Moves the pages in use to the lowest numbers and returns how many there are: pages from there on hold
        nothing. Page tables handed out before are stale afterwards."""
        used = self.num_pages - len(self._free)
        holes = sorted(p for p in self._free if p < used)
        high = [p for p in range(used, self.num_pages) if self._refs[p]]
        move = dict(zip(high, holes))
        if move:  # before anything changes: the call may raise
            msa.msa_cache_copy_pages(self.dims, list(move), list(move.values()), self.k_pool, self.v_pool, self.k_idx_pool,
                                     stream=stream)
        for s in self._seqs.values():
            s[0] = [move.get(p, p) for p in s[0]]
        for a, b in move.items():
            self._refs[b], self._refs[a] = self._refs[a], 0
        self._free = list(range(self.num_pages - 1, used - 1, -1))
        return used
