"""Rotary positions, a paged cache and the attention of drafted token trees: cases, plain forms and 64-bit values.

Five operators of the serving and training path around the sparse attention layer:

  rope    rotary positions of Q, K, Q_idx and K_idx (training and prefill), and their gradient
  append  new (or accepted drafted) tokens written into the pages of the K / V / K_idx caches
  copy    pages of the caches copied (a forked sequence's partly filled page, a compacted pool)
  select  block selection for a tree of drafted tokens over the paged index-key cache
  attend  sparse attention of a tree of drafted tokens over the paged cache and its own ancestors

A tree has T drafted tokens a sequence; node n's parent is parents[n] < n, or -1 where it follows the
cache directly. Node n at depth e sits at position cache_len + e and sees the cache and its ancestors
and itself, at positions cache_len .. cache_len + e: what a decode step would see after that path.

`run` computes an operator in elementary torch operations in 32 bits, or, where `own` is true, makes
the framework's calls. `exact` computes the same values in 64 bits, one node or head at a time.
"""
import math

import torch

own = False

DEV = "cuda"
MSA = dict(H_q=64, H_kv=4, d=128, d_idx=64, block_k=128, topk=16)  # the layer's main configuration
TINY = dict(H_q=4, H_kv=2, d=64, d_idx=32, block_k=32, topk=4)     # its smallest one


def listed():
    return [
        # rotary positions of a 32768-token prefill chunk far into a long context (full head, halves)
        dict(MSA, name="rope_prefill_32k", op="rope", back=False, tokens=32768, start=917504, rot=128, rot_idx=64,
             interleaved=False, scaling="yarn", dtype="bf16", out="bf16"),
        # gradients of a training step of odd length: fp32 dQ, dK, dQ_idx, dK_idx, part of the head, interleaved
        dict(MSA, name="rope_grad_8k", op="rope", back=True, tokens=8191, start=0, rot=64, rot_idx=32,
             interleaved=True, scaling="none", dtype="fp32", out="fp32"),
        # one decode step of a small batch: latency
        dict(MSA, name="rope_decode_16", op="rope", back=False, tokens=16, start=262143, rot=128, rot_idx=64,
             interleaved=False, scaling="linear", dtype="bf16", out="bf16"),
        # prefill chunks of 16 sequences into their pages, ragged
        dict(MSA, name="append_prefill_16x1k", op="append", B=16, L=4096, T=1024, take=False),
        # the accepted drafted tokens of 64 sequences: latency
        dict(MSA, name="append_accepted_64", op="append", B=64, L=2000, T=16, take=True),
        # a pool compacted, or many sequences forked: large copies
        dict(MSA, name="copy_1531_pages", op="copy", pages=4096, n=1531),
        # one sequence forked: its last page
        dict(MSA, name="copy_3_pages", op="copy", pages=64, n=3),
        # selection for 16 drafted tokens in each of 16 sequences of up to 262144 cached tokens
        dict(MSA, name="select_16x256k_t16", op="select", B=16, L=262144, T=16),
        # a wide tree over 8 mid-length sequences
        dict(MSA, name="select_8x50k_t64", op="select", B=8, L=50001, T=64),
        # wide trees over 16 sequences: the attention's largest case
        dict(MSA, name="attend_16x64k_t64", op="attend", B=16, L=65536, T=64),
        # short chains, the usual speculative step
        dict(MSA, name="attend_16x100k_t8", op="attend", B=16, L=99999, T=8),
        # one short sequence with one drafted token: latency
        dict(MSA, name="attend_1x3k_t1", op="attend", B=1, L=3001, T=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    """One more case: head layouts, block sizes, lengths and directions over the operators' ranges."""
    op = rng.choice(["rope", "append", "copy", "select", "attend"])
    H_kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([g for g in (1, 2, 4, 8, 16, 32) if g * H_kv <= 64])
    c = dict(H_q=G * H_kv, H_kv=H_kv, d=rng.choice([64, 128]), d_idx=rng.choice([32, 64]),
             block_k=rng.choice([32, 64, 128]), topk=rng.randint(1, 16), op=op)
    if op == "rope":
        back = rng.random() < 0.5
        dtype = rng.choice(["bf16", "fp32"])
        c |= dict(back=back, tokens=_log(rng, 1, 32768 if dtype == "bf16" else 12000), start=rng.choice([0, _log(rng, 1, 1 << 20)]),
                  rot=2 * rng.randint(1, c["d"] // 2) if rng.random() < 0.3 else rng.choice([c["d"], c["d"] // 2]),
                  rot_idx=rng.choice([c["d_idx"], c["d_idx"] // 2]), interleaved=rng.random() < 0.5,
                  scaling=rng.choice(["none", "linear", "ntk", "yarn"]), dtype=dtype,
                  out=dtype if not back else rng.choice(["bf16", "fp32"]))
    elif op == "append":
        B = _log(rng, 1, 64)
        take = rng.random() < 0.5
        T = _log(rng, 1, 64 if take else 16384 // B)
        c |= dict(B=B, T=T, L=T + _log(rng, 1, 4000), take=take)
    elif op == "copy":
        pages = _log(rng, 8, 4096)
        c |= dict(pages=pages, n=_log(rng, 1, pages // 3))
    else:
        T = _log(rng, 1, 64)
        B = _log(rng, 1, 16)
        if op == "select":
            top, most = 8000 * c["block_k"], 1 << 22 if T * H_kv <= 64 else 1 << 19
        else:
            B = max(1, min(B, 4096 // (T * H_kv)))
            top, most = 65536, 1 << 20
        c |= dict(B=B, T=T, L=_log(rng, 1, max(1, min(top, most // B))))
    return c


# ------------------------------------------------------------------------------------------- inputs
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _inv_freq(rot, scaling, base=10000.0, factor=8.0, orig=131072):
    """Inverse frequencies in 64 bits and the amplitude of the usual forms for long contexts."""
    i = torch.arange(0, rot, 2, dtype=torch.float64) / rot
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** -i
    amp = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        dim = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        amp = 0.1 * math.log(factor) + 1
    return f.to(DEV), amp


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _grid(g, *shape):
    """Index vectors on a grid of 1/16 up to 4, exact in bf16: every product and every sum of a score
    is exact in 32 bits in any order, so block maxima and their ties do not depend on the order."""
    return (torch.randn(*shape, generator=g, device=DEV).clamp(-4, 4) * 16).round().div(16).to(torch.bfloat16)


def _paged(c, g, lens_from, T_room):
    """A page table over a shuffled pool, and ragged cache lengths."""
    B, bk = c["B"], c["block_k"]
    cols = -(-(c["L"] + T_room) // bk)
    pages = B * cols + 3
    table = torch.randperm(pages, generator=g, device=DEV)[:B * cols].view(B, cols).to(torch.int32)
    lens = torch.randint(lens_from, c["L"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    lens[0] = c["L"]
    return pages, cols, table, lens


def _tree(c, g):
    """Parents below each node's own index, mostly near (long paths), and ragged node counts."""
    B, T = c["B"], c["T"]
    n = torch.arange(T, device=DEV)
    back = (torch.rand(B, T, generator=g, device=DEV) ** 2 * 6).long() + 1
    parents = (n - back).clamp(min=-1).to(torch.int32)
    n_nodes = torch.randint((T + 1) // 2, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    n_nodes[0] = T
    return parents, n_nodes


def _seen(parents):
    """Truth [B, T, T]: node n sees drafted node a (its ancestors and itself)."""
    B, T = parents.shape
    up = torch.zeros(B, T, T + 1, device=DEV, dtype=torch.float32)
    up.scatter_(2, torch.where(parents < 0, T, parents).long().unsqueeze(-1), 1.0)
    up = up[:, :, :T]
    reach = torch.eye(T, device=DEV).expand(B, T, T) + up
    reach = (reach @ reach).clamp(max=1)  # paths of up to 2, 4, 8, ... 64 steps
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    return reach > 0


def _node_blocks(c, seen, lens):
    """Each node's depth and local block."""
    depth = seen.sum(-1) - 1
    return depth, (lens[:, None] + depth) // c["block_k"]


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    H_q, H_kv, d, di, bk, k = (c[x] for x in ("H_q", "H_kv", "d", "d_idx", "block_k", "topk"))
    s = dict(c)
    if c["op"] == "rope":
        n, dt = c["tokens"], _dt(c["dtype"])
        s["x"] = [_normal(g, n, H_q, d, dtype=dt), _normal(g, n, H_kv, d, dtype=dt),
                  _normal(g, n, H_kv, di, dtype=dt), _normal(g, n, 1, di, dtype=dt)]
        f, amp = _inv_freq(c["rot"], c["scaling"])
        fi, ampi = _inv_freq(c["rot_idx"], c["scaling"])
        s["freqs"] = [(f, amp), (f, amp), (fi, ampi), (fi, ampi)]
        s["positions"] = c["start"] + torch.arange(n, device=DEV, dtype=torch.int32)
    elif c["op"] == "append":
        B, T = c["B"], c["T"]
        room = c["L"] - T
        s["pages"], cols, s["table"], _ = _paged(c, g, 1, 0)
        s["lens"] = torch.randint(0, room + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["n_new"] = torch.randint((T + 1) // 2, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["n_new"][0] = T
        s["rows"] = None
        if c["take"]:  # an accepted path: ascending node numbers, each row its own
            order = torch.rand(B, T, generator=g, device=DEV).argsort(1)
            live = torch.arange(T, device=DEV) < s["n_new"][:, None]
            s["rows"] = torch.where(live, order, T).sort(1).values.clamp(max=T - 1).to(torch.int32)
        s["new"] = [_normal(g, B, T, H_kv, d), _normal(g, B, T, H_kv, d), _normal(g, B, T, di)]
        s["pools"] = [_normal(g, s["pages"], bk, H_kv, d), _normal(g, s["pages"], bk, H_kv, d), _normal(g, s["pages"], bk, di)]
    elif c["op"] == "copy":
        order = torch.randperm(c["pages"], generator=g, device=DEV).to(torch.int32)
        s["src"], s["dst"] = order[:c["n"]].contiguous(), order[-c["n"]:].contiguous()
        s["pools"] = [_normal(g, c["pages"], bk, H_kv, d), _normal(g, c["pages"], bk, H_kv, d), _normal(g, c["pages"], bk, di)]
    else:
        B, T = c["B"], c["T"]
        s["pages"], cols, s["table"], s["lens"] = _paged(c, g, (c["L"] + 1) // 2, T)
        s["parents"], s["n_nodes"] = _tree(c, g)
        if c["op"] == "select":
            s["q_idx"] = _grid(g, B, T, H_kv, di)
            s["k_idx"], s["k_idx_pool"] = _grid(g, B, T, di), _grid(g, s["pages"], bk, di)
        else:
            s["q"], s["k"], s["v"] = _normal(g, B, T, H_q, d), _normal(g, B, T, H_kv, d), _normal(g, B, T, H_kv, d)
            s["k_pool"], s["v_pool"] = _normal(g, s["pages"], bk, H_kv, d), _normal(g, s["pages"], bk, H_kv, d)
            s["blocks"] = _lists(c, g, s["parents"], s["n_nodes"], s["lens"])
    return s


def _shared(c):
    """Blocks that the nodes of one tree choose from in a (sequence, group): their queries are near."""
    return c["topk"] + 2 * (c["T"].bit_length() - 1)


def _lists(c, g, parents, n_nodes, lens):
    """Selected blocks as a selection gives them: up to topk of the blocks that the tree's nodes share,
    the cache's last block where the path has left it, and the local block; ascending, -1 padded."""
    B, T, H_kv, k, bk = c["B"], c["T"], c["H_kv"], c["topk"], c["block_k"]
    full = lens // bk                                            # complete blocks of the cache
    _, local = _node_blocks(c, _seen(parents), lens)
    cols = int(-(-(c["L"]) // bk)) + 1
    far = torch.rand(B, H_kv, cols, generator=g, device=DEV)
    far = torch.where(torch.arange(cols, device=DEV) < full[:, None, None], far, 2.0)
    pool = far.sort(-1).indices[..., :min(_shared(c), cols)]      # [B, H_kv, U], complete blocks first
    U = pool.shape[-1]
    live = torch.arange(U, device=DEV) < full[:, None, None]
    want = torch.rand(B, T, H_kv, U, generator=g, device=DEV)
    want = torch.where(live[:, None], want, 2.0)
    kk = min(k, U)
    pick = want.sort(-1).indices[..., :kk]
    ids = pool[:, None].expand(B, T, H_kv, U).gather(-1, pick)
    j = torch.arange(kk, device=DEV)
    past = (local > full[:, None])[:, :, None, None]             # the path has left the cache's last block
    ids = torch.where((j < full[:, None, None, None]) & ~(past & (j == k - 1)), ids, 1 << 30)
    last = torch.where(past, full[:, None, None, None].expand(B, T, H_kv, 1), 1 << 30)
    ids = torch.cat([ids, last, local[:, :, None, None].expand(B, T, H_kv, 1)], -1).sort(-1).values
    ids = torch.nn.functional.pad(ids, (0, max(0, k + 1 - ids.shape[-1])), value=1 << 30)[..., :k + 1]
    ids = torch.where((ids == 1 << 30) | (torch.arange(T, device=DEV) >= n_nodes[:, None])[:, :, None, None], -1, ids)
    return ids.to(torch.int32).contiguous()


# ---------------------------------------------------------------------------------------- the passes
def run(state):
    s = state
    if own:
        import block_sparse_attention_idx_b200 as msa

        if s["op"] == "rope":
            turn = msa.msa_rope_bwd if s["back"] else msa.msa_rope_fwd
            return turn(s["x"], s["freqs"], s["positions"], interleaved=s["interleaved"], out_dtype=_dt(s["out"]))
        N = 0 if s["op"] == "copy" else s["table"].shape[1] * s["block_k"]
        dims = msa.MsaDims(s.get("B", 1), N or s["block_k"], s["H_q"], s["H_kv"], s["d"], s["d_idx"], s["block_k"], s["topk"])
        if s["op"] == "copy":
            msa.msa_cache_copy_pages(dims, s["src"], s["dst"], *s["pools"])
            return s["pools"]
        pages = msa.MsaPages(s["table"], s["lens"])
        if s["op"] == "append":
            msa.msa_cache_append(dims, pages, *s["new"], *s["pools"], s["n_new"], rows=s["rows"])
            return s["pools"]
        tree = msa.MsaTree(s["parents"], s["n_nodes"])
        if s["op"] == "select":
            return msa.msa_tree_index_topk(dims, pages, tree, s["q_idx"], s["k_idx"], s["k_idx_pool"], want_margin=True)
        return msa.msa_tree_sparse_attn(dims, pages, tree, s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["blocks"], want_lse=True,
                                        out_dtype=torch.bfloat16)
    return {"rope": _rope, "append": _append, "copy": _copy, "select": _select, "attend": _attend}[s["op"]](s)


def _rotate(x, freq, positions, interleaved, back, out):
    f, amp = freq
    r = 2 * f.numel()
    angle = positions.double()[:, None] * f                      # 64 bits: far positions lose the angle in 32
    cos, sin = (angle.cos() * amp).float()[:, None], (angle.sin() * (-amp if back else amp)).float()[:, None]
    y = x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, y[..., r:]], -1).to(out)


def _rope(s):
    return [_rotate(x, f, s["positions"], s["interleaved"], s["back"], _dt(s["out"])) for x, f in zip(s["x"], s["freqs"])]


def _append(s):
    T, bk = s["T"], s["block_k"]
    at = torch.minimum(torch.arange(T, device=DEV), s["n_new"][:, None] - 1).long()  # past the last: the last again
    slot = s["lens"][:, None] + at
    page = s["table"].long().gather(1, slot // bk)
    row = at if s["rows"] is None else s["rows"].long().gather(1, at)
    b = torch.arange(s["B"], device=DEV)[:, None]
    s["pools"][0][page, slot % bk] = s["new"][0][b, row]
    s["pools"][1][page, slot % bk] = s["new"][1][b, row]
    s["pools"][2][page, slot % bk] = s["new"][2][b, row]
    return s["pools"]


def _copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    s["pools"][0][dst] = s["pools"][0][src]
    s["pools"][1][dst] = s["pools"][1][src]
    s["pools"][2][dst] = s["pools"][2][src]
    return s["pools"]


def _select(s):
    B, T, H_kv, bk, k = s["B"], s["T"], s["H_kv"], s["block_k"], s["topk"]
    low = -math.inf
    seen = _seen(s["parents"])
    depth, local = _node_blocks(s, seen, s["lens"])
    cols = s["table"].shape[1]
    keys = s["k_idx_pool"][s["table"].long()].view(B, cols * bk, -1).float()
    q = s["q_idx"].float()
    score = torch.einsum("btgc,blc->btgl", q, keys)
    score.masked_fill_((torch.arange(cols * bk, device=DEV) >= s["lens"][:, None])[:, None, None], low)
    best = torch.cat([score.view(B, T, H_kv, cols, bk).amax(-1), score.new_full((B, T, H_kv, 3), low)], -1)
    mine = torch.einsum("btgc,bac->btga", q, s["k_idx"].float()).masked_fill(~seen[:, :, None], low)
    at = local[:, None, None].expand(B, T, H_kv, T)              # the drafted tokens' own blocks
    best = best.scatter_reduce(-1, at, mine, "amax")
    blk = torch.arange(best.shape[-1], device=DEV)
    best = torch.where(blk < local[:, :, None, None], best, low)
    best = torch.cat([best, best.new_full((B, T, H_kv, k + 1), low)], -1)
    order = best.sort(stable=True, dim=-1, descending=True)      # ties: the lowest block first
    none = 1 << 30
    ids = torch.where(torch.arange(k, device=DEV) < local[:, :, None, None], order.indices[..., :k], none)
    ids = torch.cat([ids, local[:, :, None, None].expand(B, T, H_kv, 1)], -1).sort(-1).values
    gone = (torch.arange(T, device=DEV) >= s["n_nodes"][:, None])[:, :, None, None]
    margin = (order.values[..., k - 1] - order.values[..., k]) / math.sqrt(s["d_idx"])   # of the k-th block over the next
    margin = torch.where((local[:, :, None] > k) & ~gone[..., 0], margin, math.inf)
    return torch.where((ids == none) | gone, -1, ids).to(torch.int32), margin


def _attend(s):
    B, T, H_q, H_kv, bk, d = (s[x] for x in ("B", "T", "H_q", "H_kv", "block_k", "d"))
    G = H_q // H_kv
    seen = _seen(s["parents"])
    depth, _ = _node_blocks(s, seen, s["lens"])
    blocks = s["blocks"].long()
    pos = (blocks[..., None] * bk + torch.arange(bk, device=DEV)).flatten(-2)     # [B, T, H_kv, J]
    lens = s["lens"].long()[:, None, None, None]
    there = (blocks >= 0)[..., None].expand(*blocks.shape, bk).flatten(-2) & (pos <= lens + depth[:, :, None, None])
    # cached positions through the page table, later ones through the node's own path
    page = s["table"].long()[:, None, None].expand(B, T, H_kv, -1).gather(-1, (pos // bk).clamp(0, s["table"].shape[1] - 1))
    cached = page * bk + pos % bk
    path = torch.zeros(B, T, T, device=DEV, dtype=torch.long)                      # node at each depth of node n's path
    path.scatter_reduce_(2, torch.where(seen, depth[:, None].expand(B, T, T), 0), torch.where(seen, torch.arange(T, device=DEV), 0), "amax")
    step = (pos - lens).clamp(0, T - 1)
    drafted = path[:, :, None].expand(B, T, H_kv, T).gather(-1, step) + T * torch.arange(B, device=DEV)[:, None, None, None]
    g = torch.arange(H_kv, device=DEV)[:, None]
    old = (pos < lens)[..., None]
    cached, drafted = torch.where(pos < lens, cached, 0), torch.where(there, drafted, 0)
    q = s["q"].view(B, T, H_kv, G, d).float()
    key = torch.where(old, s["k_pool"].view(-1, H_kv, d)[cached, g], s["k"].view(-1, H_kv, d)[drafted, g]).float()
    logit = (q @ key.transpose(-1, -2)) / math.sqrt(d)
    logit.masked_fill_(~there[:, :, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = (logit - top.clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = p.sum(-1, keepdim=True)
    del key
    val = torch.where(old, s["v_pool"].view(-1, H_kv, d)[cached, g], s["v"].view(-1, H_kv, d)[drafted, g]).float()
    out = (p @ val) / torch.where(total > 0, total, 1.0)
    return out.view(B, T, H_q, d).to(torch.bfloat16), (top + total.log()).view(B, T, H_q)


# ------------------------------------------------------------------------------------------ the floor
def _expect(c):
    """Mean cache length and node count of a case's ragged sequences."""
    B = c["B"]
    low = (c["L"] + 1) // 2
    lens = (c["L"] + (B - 1) * (low + c["L"]) / 2) / B
    nodes = (c["T"] + (B - 1) * ((c["T"] + 1) // 2 + c["T"]) / 2) / B
    return lens, nodes


def work(case):
    c = case
    H_q, H_kv, d, di, bk, k = (c[x] for x in ("H_q", "H_kv", "d", "d_idx", "block_k", "topk"))
    token = (2 * H_kv * d + di) * 2                              # bytes of one cached token
    if c["op"] == "rope":
        each = (H_q + H_kv) * d + (H_kv + 1) * di
        size = {"bf16": 2, "fp32": 4}
        turned = (H_q + H_kv) * c["rot"] + (H_kv + 1) * c["rot_idx"]
        return {"bytes": c["tokens"] * (each * (size[c["dtype"]] + size[c["out"]]) + 4), "flops": 3 * c["tokens"] * turned}
    if c["op"] == "append":
        return {"bytes": 2 * token * c["T"] * (0.75 * (c["B"] - 1) + 1), "flops": 0}
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * bk * token, "flops": 0}
    lens, nodes = _expect(c)
    B, T = c["B"], c["T"]
    if c["op"] == "select":
        return {"bytes": B * (lens * di * 2 + T * (H_kv + 1) * di * 2 + T * H_kv * (k + 2) * 4),
                "flops": 2.0 * B * nodes * H_kv * lens * di}
    full = lens // bk
    U = min(_shared(c), full)
    kept = min(k, U)
    distinct = U * (1 - (1 - kept / U) ** nodes) if U else 0
    row = distinct * bk + lens % bk + T
    return {"bytes": B * (H_kv * row * d * 4 + T * H_q * (d * 4 + 4) + T * H_kv * (k + 1) * 4),
            "flops": 4.0 * d * B * nodes * H_q * (kept * bk + lens % bk)}


# ------------------------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rope":
        return [_turned(x, f, c, s["positions"]) for x, f in zip(s["x"], s["freqs"])]
    if c["op"] in ("append", "copy"):
        return [_moved(c, s, i) for i in range(3)]
    if c["op"] == "select" and c["B"] * c["T"] * c["L"] * c["H_kv"] > 1 << 31:
        return None
    return _exact_select(c, s) if c["op"] == "select" else _exact_attend(c, s)


def _turned(x, freq, c, positions):
    f, amp = freq
    r = 2 * f.numel()
    z = x.double()
    pairs = z[..., :r].unflatten(-1, (r // 2, 2)) if c["interleaved"] else z[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    w = torch.polar(torch.full((positions.numel(), 1, r // 2), amp, device=DEV, dtype=torch.float64),
                    (positions.double()[:, None, None] * f) * (-1 if c["back"] else 1))
    t = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    z[..., :r] = t.flatten(-2) if c["interleaved"] else t.transpose(-1, -2).flatten(-2)
    return z


def _moved(c, s, i):
    pool = s["pools"][i].clone()
    if c["op"] == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[b] = s["pools"][i][a]
        return pool.double()
    flat = pool.view(-1, *pool.shape[2:])
    for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["n_new"].tolist())):
        slots = torch.arange(n, n + m, device=DEV)
        rows = torch.arange(m, device=DEV) if s["rows"] is None else s["rows"][b, :m].long()
        flat[s["table"][b].long()[slots // c["block_k"]] * c["block_k"] + slots % c["block_k"]] = s["new"][i][b][rows]
    return pool.double()


def _paths(s, b):
    up = s["parents"][b].tolist()
    made = []
    for n in range(int(s["n_nodes"][b])):
        made.append((made[up[n]] if up[n] >= 0 else []) + [n])
    return made


def _exact_select(c, s):
    B, T, bk, k = c["B"], c["T"], c["block_k"], c["topk"]
    out = torch.full((B, T, c["H_kv"], k + 1), -1, dtype=torch.int32)
    margin = torch.full((B, T, c["H_kv"]), math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(s["lens"][b])
        old = s["k_idx_pool"][s["table"][b].long()].flatten(0, 1)[:n].double()
        for t, path in enumerate(_paths(s, b)):
            keys = torch.cat([old, s["k_idx"][b, path].double()])
            local = (keys.shape[0] - 1) // bk
            if local:
                top = (s["q_idx"][b, t].double() @ keys[:local * bk].T).view(-1, local, bk).amax(-1)
                top, first = top.sort(stable=True, dim=-1, descending=True)
                if local > k:
                    margin[b, t] = (top[:, k - 1] - top[:, k]) * c["d_idx"] ** -0.5
                first = first[:, :k].sort(-1).values.cpu()
                out[b, t, :, :first.shape[1]] = first
            out[b, t, :, min(k, local)] = local
    return out.to(DEV), margin


def _exact_attend(c, s):
    B, T, H_q, H_kv, d, bk = (c[x] for x in ("B", "T", "H_q", "H_kv", "d", "block_k"))
    G = H_q // H_kv
    out = torch.zeros(B, T, H_q, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, H_q), -math.inf, dtype=torch.float64, device=DEV)
    pool = s["k_pool"].view(-1, H_kv, d), s["v_pool"].view(-1, H_kv, d)
    blocks = s["blocks"].tolist()
    for b in range(B):
        n, table = int(s["lens"][b]), s["table"][b].tolist()
        for t, path in enumerate(_paths(s, b)):
            for g in range(H_kv):
                want = [j for x in blocks[b][t][g] if x >= 0 for j in range(x * bk, min((x + 1) * bk, n + len(path)))]
                if not want:
                    continue
                old = torch.tensor([table[j // bk] * bk + j % bk for j in want if j < n], dtype=torch.long, device=DEV)
                new = torch.tensor([path[j - n] for j in want if j >= n], dtype=torch.long, device=DEV)
                key = torch.cat([pool[0][old, g], s["k"][b][new, g]]).double()
                val = torch.cat([pool[1][old, g], s["v"][b][new, g]]).double()
                z = s["q"][b, t, g * G:(g + 1) * G].double() @ key.T * d ** -0.5
                lse[b, t, g * G:(g + 1) * G] = z.logsumexp(-1)
                out[b, t, g * G:(g + 1) * G] = z.softmax(-1) @ val
    return out, lse
