// Sparse attention of drafted-token trees over a paged cache. Row (node, head h of group r) attends the
// tokens of its virtual sequence (the cache, its ancestors, itself) that lie in the blocks of its list
// blocks[b, node, r, :]: softmax(q . k * scale) v.
//
// Query-outer: one CTA holds 128 rows (128 / G nodes with the G heads of one group) and walks the union of their
// selected pages, so that a page that several nodes chose, which is the rule (their queries are near), is loaded once
// per CTA and no partial outputs are spilled; a node that did not choose a page is masked there. The union is a bitmap
// over the sequence's blocks in shared memory, its order the block order, each entry with the set of nodes that chose
// it. Keys go in tiles of 128: first the drafted tokens, masked to each node's ancestors in its selected blocks, whose
// loads run while the union is built, then the pages, 128 / block_k a tile.
//
// Per tile: S = Q K^T (tcgen05, M = N = 128) in TMEM; two threads share a row, 64 columns each: maximum, exponentials
// (base 2) and sums in fp32, P as bf16 over S; O += P V accumulates in TMEM. The running maximum is only raised, and O
// rescaled, when a row's maximum grows by more than 2^8: exponents stay far inside fp32 and bf16, and most tiles
// rescale nothing. P is rounded to bf16 for the product (whose operands share V's type), each weight by a factor
// 1 + e, |e| <= 2^-8. O is divided by the fp32 sum of the rounded weights, so that the weights that were used sum to one and
// the error is sum w e (v - o): it follows the spread of the values, not their size (dividing by the sum of the unrounded
// ones took 134 us instead of 138 at 64 nodes over 16 x 65536 tokens, and moved outputs of values around 64 by up to 0.06). The LSE
// takes the sum of the fp32 exponentials. The products accumulate in fp32.
//
// A CTA is a chain: S, exponentials, PV, next S. Two CTAs share an SM (256 TMEM columns, 113 KB and 96 registers a
// thread each), so that one's products, loads, list building and output run under the other's exponentials. K and V
// have one buffer each: K of the next tile arrives during this tile's exponentials, V during the next tile's. The last
// wave of CTAs, if it would fill at most half of the device, splits its unions over several CTAs, merged by
// k_tree_combine: 64 nodes over 16 x 65536 tokens (408 items of 128 rows, 30 tiles each; 64 query heads in 4 groups,
// d = 128) took 132 us instead of 144 by that, and a few nodes of a long tree take what they would take alone.
//
// Bound, 64 nodes (140 us, 1.09 TB/s and 380 TFLOP/s): the chain. Before the rounded weights had their own sum (134 us)
// a tile took 3700 cycles, 2030 of them the exponentials and what is around them (1024 on the MUFU, which both CTAs share),
// 1650 from P to the next S (1024 of products: 128 x 128 x 16 take 64 cycles with both operands in shared memory); the
// tensor pipe is busy 39 % of the time, the MUFU 32 %. At 8 nodes a sequence (256 CTAs of 6 tiles: 39 us with the merge) it
// waits for pages that nobody has read before (2300 cycles a tile for V), and list building and output cost 9 us of a CTA's
// 28.
#include <type_traits>

#include "msa_tree.cuh"

namespace msa {

namespace {

constexpr int kRows = 128;
constexpr int kMaxEntries = kTreeMaxT * 17;  // union of a CTA's lists
constexpr int kWords = kTreeMaxBlocks / 32;

constexpr int kAttnThreads = 320;  // warps 0-7 softmax, 8 TMA, 9 MMA

// What only the list building needs; it lies in V's buffer, behind the 64 rows that the drafted tokens' load fills
// meanwhile (in the first 64-column half).
struct TreeLists {
    unsigned long long anc[64];       // ancestors of a node
    unsigned long long in_block[4];   // nodes whose position lies in block len / block_k + i
    int local[64];                    // local block of a node
    uint32_t late[64];                // blocks >= len / block_k in a node's list
    uint32_t bits[kWords];            // the union
    int before[kWords];               // entries before a word's
};

template <int D>
struct TreeAttnSmem {
    alignas(1024) uint8_t q[kRows * D * 2];
    alignas(1024) uint8_t k[kTile * D * 2];  // with v, at the end: outputs on their way out
    alignas(1024) uint8_t v[kTile * D * 2];
    unsigned long long mask[kMaxEntries];  // nodes of the CTA that chose the entry
    unsigned long long draft[64];          // drafted tokens that a node attends
    int page[kMaxEntries];
    float row_max[2][kRows], row_sum[2][kRows];  // exchange between the two threads of a row
    uint64_t k_full, k_empty, v_full, v_empty, s_full, p_ready, pv_done, drain;
    int total, partial;
    uint32_t tmem_base;
};
static_assert(sizeof(TreeAttnSmem<128>) + 1024 <= 113 * 1024, "two CTAs share an SM");
static_assert(sizeof(TreeLists) <= 64 * 128, "the lists fit V's rows 64 .. 127");

// Three-input maximum that keeps a NaN.
__device__ __forceinline__ float max3n(float a, float b, float c) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// An item is 128 rows: the nodes ct * 128/G .. of sequence b, group r. Items without a node that exists are left out
// (unless a sequence has only one item per group). The device runs `slots` CTAs at once, so the items' last, part-filled
// wave is the one whose length counts: its `rem` items are split over `splits` CTAs each, as many as the slots hold.
struct TreeUnit {
    int b, r, ct;
    int split, splits;
    int part;  // of the partial outputs, where splits > 1: split i of the j-th split item has part i * (split items) + j
};
__device__ __forceinline__ int tree_items(const TreeArgs& a, int b) {  // per group of sequence b
    const int sh = 7 - a.lg_g;
    return b >= a.B ? 0 : a.T <= (kRows >> a.lg_g) ? 1 : (tree_nodes(a, b) + (1 << sh) - 1) >> sh;
}
// Called by whole warps. What CTA `unit` does; false if nothing. Items are ordered by sequence, group and node:
// neighbours share pages. count: the split items and their CTAs.
__device__ __forceinline__ bool tree_unit(const TreeArgs& a, int unit, TreeUnit* u, int2* count) {
    const int lane = threadIdx.x & 31;
    const bool even = a.T <= (kRows >> a.lg_g);  // one item per sequence and group
    // items per group of the sequences lo .. lo + n - 1, `per` of them a lane: a lane's, and up to and with the lane's
    int lo = 0, n = a.B, per, mine, incl;
    auto count_items = [&] {
        per = (n + 31) / 32;
        mine = 0;
        for (int i = lane * per; i < min(n, (lane + 1) * per); ++i) mine += tree_items(a, lo + i);
        incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
    };
    int live = a.B;
    if (!even) {
        count_items();
        live = __shfl_sync(0xffffffffu, incl, 31);
    }
    live *= a.H_kv;
    const int base = live < a.slots ? 0 : live / a.slots * a.slots, rem = live - base;
    const int splits = rem > 0 ? max(1, min(a.max_splits, a.slots / rem)) : 1;
    *count = make_int2(rem, splits);
    int item = unit;
    u->split = 0, u->splits = 1, u->part = 0;
    if (unit >= base) {
        if (unit - base >= rem * splits) return false;
        u->part = unit - base, u->splits = splits, u->split = u->part / rem, item = unit - u->split * rem;
    }
    if (even) {
        u->b = item / a.H_kv, u->r = item - u->b * a.H_kv, u->ct = 0;
        return true;
    }
    for (int before = 0;;) {  // to the lane that has the item, then among its sequences
        const int l = __ffs(__ballot_sync(0xffffffffu, (before + incl) * a.H_kv > item)) - 1;
        before += __shfl_sync(0xffffffffu, incl - mine, l);
        lo += l * per;
        if (per == 1) {
            const int cts = __shfl_sync(0xffffffffu, mine, l), at = item - before * a.H_kv;
            u->b = lo, u->r = at / cts, u->ct = at - u->r * cts;
            return true;
        }
        n = min(per, n - l * per);
        count_items();
    }
}

// Zeros and LSE -inf for the rows of nodes n0 .. that lie in T.
__device__ __forceinline__ void tree_zero_rows(const TreeArgs& a, int b, int r, int n0) {
    const int lg = a.lg_g, rows = min(kRows, (a.T - n0) << lg), pieces = a.d / 8;
    auto out_row = [&](int i) { return ((int64_t)b * a.T + n0 + (i >> lg)) * a.H_q + (r << lg) + (i & ((1 << lg) - 1)); };
    for (int i = threadIdx.x; a.lse && i < rows; i += blockDim.x) a.lse[out_row(i)] = -INFINITY;
    for (int i = threadIdx.x; i < rows * pieces; i += blockDim.x) {
        const int64_t o = out_row(i / pieces) * a.d + (i % pieces) * 8;
        if (a.out_bf16) {
            *reinterpret_cast<uint4*>(a.out_bf16 + o) = make_uint4(0, 0, 0, 0);
        } else {
            *reinterpret_cast<uint4*>(a.out + o) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(a.out + o + 4) = make_uint4(0, 0, 0, 0);
        }
    }
}

// One warp: half `hf` of the output columns of row `ri` of a CTA, by the definition, from the tokens that the row sees
// among the drafted ones (if the CTA has them) and the entries [e_lo, e_hi) of the union. For rows whose product is not
// finite: a weight of zero times an infinity or NaN in V (of a token that another node chose), or values so large that a
// weight of up to 2^8 overflowed. lse2: the row's base-2 log-sum-exp over these tokens, so that no weight exceeds 1. A row
// of 2176 tokens takes 0.3 ms, one warp's chain of loads; looking for such rows costs 2 us of the 140 at 64 nodes over
// 16 x 65536 tokens.
template <int D, int BK>
__device__ __noinline__ void tree_row_by_tokens(const TreeArgs& a, const TreeAttnSmem<D>& s, int b, int r, int ri, int hf, bool drafted,
                                                int e_lo, int e_hi, int last_entry_keys, float lse2, float* out,
                                                __nv_bfloat16* out_bf16) {
    constexpr int KQ = D / 32, KV = D / 64, U = 4;  // elements of a key, of a value that a lane holds; tokens under way
    const int lane = lane_id(), nl = ri >> a.lg_g;
    const float sl2 = a.scale * 1.4426950408889634f;
    float qf[KQ], acc[KV];
#pragma unroll
    for (int x = 0; x < KQ; ++x) {
        const int c = lane * KQ + x;
        qf[x] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(s.q + (c / 64) * (kTile * 128) + swz(ri, (c % 64) * 2, 128)));
    }
#pragma unroll
    for (int x = 0; x < KV; ++x) acc[x] = 0.f;
    auto tokens = [&](const __nv_bfloat16* k, const __nv_bfloat16* v, int64_t first, int n, unsigned long long which) {
        for (int t0 = 0; t0 < n; t0 += U) {
            float dot[U], vf[U][KV];
#pragma unroll
            for (int t = 0; t < U; ++t) {
                const int64_t at = ((first + min(t0 + t, n - 1)) * a.H_kv + r) * D;
                dot[t] = 0.f;
#pragma unroll
                for (int x = 0; x < KQ; ++x) dot[t] = fmaf(qf[x], __bfloat162float(k[at + lane * KQ + x]), dot[t]);
#pragma unroll
                for (int x = 0; x < KV; ++x) vf[t][x] = __bfloat162float(v[at + hf * (D / 2) + lane * KV + x]);
            }
#pragma unroll
            for (int t = 0; t < U; ++t) {
#pragma unroll
                for (int o = 16; o; o >>= 1) dot[t] += __shfl_xor_sync(0xffffffffu, dot[t], o);
                const float w = exp2f(fmaf(dot[t], sl2, -lse2));
                if (t0 + t < n && ((which >> ((t0 + t) & 63)) & 1)) {
#pragma unroll
                    for (int x = 0; x < KV; ++x) acc[x] = fmaf(w, vf[t][x], acc[x]);
                }
            }
        }
    };
    if (drafted) tokens(a.k, a.v, (int64_t)b * a.T, a.T, s.draft[nl]);
    for (int e = e_lo; e < e_hi; ++e)
        if ((s.mask[e - e_lo] >> nl) & 1)
            tokens(a.k_pool, a.v_pool, (int64_t)s.page[e - e_lo] * BK, e == e_hi - 1 ? last_entry_keys : BK, ~0ull);
#pragma unroll
    for (int x = 0; x < KV; ++x) {
        const int c = hf * (D / 2) + lane * KV + x;
        if (out_bf16) out_bf16[c] = __float2bfloat16_rn(acc[x]);
        else out[c] = acc[x];
    }
}

template <int D, int BK>
__global__ void __launch_bounds__(kAttnThreads, 2)
    k_tree_attn(const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                const __grid_constant__ CUtensorMap tm_kd, const __grid_constant__ CUtensorMap tm_vd,
                const __grid_constant__ TreeArgs a, const __nv_bfloat16* __restrict__ q) {
    using Sm = TreeAttnSmem<D>;
    constexpr int TPT = kTile / BK;
    constexpr int NT = kAttnThreads;
    constexpr int kTmaWarp = 8, kMmaWarp = 9;
    constexpr uint32_t kHalf = kTile * 128;  // bytes of a 64-column half of a 128-row tile
    constexpr int kColO = 128;  // TMEM columns: S (then P) at 0, O at 128
    constexpr int EPT = (kMaxEntries + NT - 1) / NT;  // list entries per thread
    extern __shared__ uint8_t tree_raw[];
    Sm& s = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(tree_raw) + 1023) & ~uintptr_t(1023));
    TreeLists& ls = *reinterpret_cast<TreeLists*>(s.v + 64 * 128);
    const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
    const int lg = a.lg_g, K1 = a.topk + 1;     // G = 2^lg heads per group
    const int per_cta = kRows >> lg;            // nodes
    auto list_of = [&](int e) { return (e * a.k1_inv) >> 16; };  // e / K1
    if (a.T > per_cta) {  // items without a node: CTA i writes the i-th of all, if it is one
        const int n_ct = (a.T + per_cta - 1) / per_cta, i = blockIdx.x;
        const int zc = i % n_ct, zr = i / n_ct % a.H_kv, zb = i / n_ct / a.H_kv;
        if (zb < a.B && zc * per_cta >= tree_nodes(a, zb)) {
            tree_zero_rows(a, zb, zr, zc * per_cta);
            if (tid == 0 && zr == 0 && zc == 0 && (tree_len(a, zb) != a.cache_len[zb] || a.n_nodes[zb] != 0))
                raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xc01);
        }
    }
    TreeUnit u;
    int2 count;
    const bool live_cta = tree_unit(a, blockIdx.x, &u, &count);
    if (tid == 0) {  // for the merge
        if (blockIdx.x == 0) *a.split_count = count;
        if (live_cta && u.splits > 1 && u.split == 0) a.split_items[u.part] = make_int4(u.b, u.r, u.ct, 0);
    }
    if (!live_cta) {
        pdl_trigger();
        return;
    }
    const int b = u.b, r = u.r, ct = u.ct, split = u.split, n0 = ct * per_cta;

    // ------------------------------------------------------------------ the union of the CTA's lists
    // Loads that depend on nothing go first: the lists (kept in registers), the parents, Q. Rows of nodes that
    // do not exist are loaded too: nothing they hold reaches another row, and they see no key.
    int id[EPT], pg[EPT];
    const int n_ent = min(per_cta, a.T - n0) * K1;
#pragma unroll
    for (int x = 0; x < EPT; ++x) {
        const int e = tid + x * NT;
        const int nl = list_of(e);
        id[x] = e < n_ent ? a.blocks[(((int64_t)b * a.T + n0 + nl) * a.H_kv + r) * K1 + e - nl * K1] : -1;
    }
    // the pages of the listed blocks, before it is known which of them count
#pragma unroll
    for (int x = 0; x < EPT; ++x)
        pg[x] = (unsigned)id[x] < (unsigned)a.cols ? a.page_table[(int64_t)b * a.cols + id[x]] : -1;
    int p0 = -1, p1 = -1;
    if (warp == kTmaWarp) {
        p0 = load_parent(a, b, lane);
        p1 = load_parent(a, b, lane + 32);
    }
    const int len = tree_len(a, b), nodes = tree_nodes(a, b);
    if (n0 >= nodes) {  // a sequence without nodes: zeros (its partial outputs are not read) and LSE -inf
        if (tid == 0 && r == 0 && split == 0 && (len != a.cache_len[b] || nodes != a.n_nodes[b]))
            raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xc01);
        if (u.splits == 1) tree_zero_rows(a, b, r, n0);
        else if (tid < a.part_rows) a.lse_part[u.part * a.part_rows + tid] = -INFINITY;
        pdl_trigger();
        return;
    }
    if (warp == kTmaWarp && elect_one()) {
        mbar_init(&s.k_full, 1);
        mbar_init(&s.k_empty, 1);
        mbar_init(&s.v_full, 1);
        mbar_init(&s.v_empty, 1);
        mbar_init(&s.s_full, 1);
        mbar_init(&s.p_ready, 8);
        mbar_init(&s.pv_done, 1);
        mbar_init(&s.drain, 1);
        fence_mbar_init();
        if (split == 0) {  // the drafted tokens' tile
            mbar_arrive_expect_tx(&s.k_full, 64u * D * 2);
            mbar_arrive_expect_tx(&s.v_full, 64u * D * 2);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                tma_load_4d(s.k + h * kHalf, &tm_kd, &s.k_full, 64 * h, r, 0, b);
                tma_load_4d(s.v + h * kHalf, &tm_vd, &s.v_full, 64 * h, r, 0, b);
            }
        }
        prefetch_tmap(&tm_kp);
        prefetch_tmap(&tm_vp);
    }
    __syncwarp();
    for (int i = tid; i < kRows * (D / 8); i += NT) {
        const int row = i / (D / 8), c = i % (D / 8), node = n0 + (row >> lg), h = row & ((1 << lg) - 1);
        const uint32_t dst = smem_u32(s.q) + (c / 8) * kHalf + swz(row, (c % 8) * 16, 128);
        const bool live = node < a.T;
        cp_async_16_zfill(dst, live ? q + (((int64_t)b * a.T + node) * a.H_q + (r << lg) + h) * D + c * 8 : q, live);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s.tmem_base, 256);
        tmem_relinquish();
    }
    for (int i = tid; i < kWords; i += NT) ls.bits[i] = 0u;
    for (int i = tid; i < kMaxEntries; i += NT) s.mask[i] = 0ull;
    if (tid < 64) ls.late[tid] = 0u;
    const int full = len / BK, npages = (len + BK - 1) / BK;  // complete pages, pages
    if (warp == kTmaWarp) {
        if (lane == 0 && r == 0 && ct == 0 && split == 0 && (len != a.cache_len[b] || nodes != a.n_nodes[b]))
            raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xc01);
        unsigned long long anc[2];
        tree_ancestors(a, nodes, p0, p1, anc, 0xc02);
        int off[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int n = lane + 32 * x, loc = (len + __popcll(anc[x]) - 1) / BK;
            ls.anc[n] = anc[x];
            ls.local[n] = loc;
            off[x] = n < nodes ? loc - full : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = __ballot_sync(0xffffffffu, off[0] == i), hi = __ballot_sync(0xffffffffu, off[1] == i);
            if (lane == 0) ls.in_block[i] = ((unsigned long long)hi << 32) | lo;
        }
    }
    __syncthreads();
    const int mine = max(0, min(per_cta, nodes - n0));  // nodes of this CTA that exist
#pragma unroll
    for (int x = 0; x < EPT; ++x) {
        const int nl = list_of(tid + x * NT);
        if (id[x] == -1 || nl >= mine) {
            id[x] = -1;
        } else if (id[x] < -1 || id[x] > ls.local[n0 + nl]) {
            raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xc03);
            id[x] = -1;
        } else {
            if (id[x] >= full) atomicOr(&ls.late[nl], 1u << (id[x] - full));
            if (id[x] < npages) {
                atomicOr(&ls.bits[id[x] >> 5], 1u << (id[x] & 31));
                if ((unsigned)pg[x] >= (unsigned)a.num_pages) {
                    raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xc04);
                    pg[x] = 0;
                }
            } else {
                id[x] = -1;
            }
        }
    }
    __syncthreads();
    if (warp == 0) {
        int sum = 0;
#pragma unroll
        for (int x = 0; x < kWords / 32; ++x) sum += __popc(ls.bits[lane * (kWords / 32) + x]);
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        int at = incl - sum;
#pragma unroll
        for (int x = 0; x < kWords / 32; ++x) {
            ls.before[lane * (kWords / 32) + x] = at;
            at += __popc(ls.bits[lane * (kWords / 32) + x]);
        }
        if (lane == 31) s.total = incl;
        if (lane == 0) s.partial = npages > full && ((ls.bits[full >> 5] >> (full & 31)) & 1);
    } else if (tid >= 64 && tid < 128) {
        // drafted tokens that a node attends: its ancestors in its selected blocks
        const int nl = tid - 64;
        unsigned long long d = 0ull;
        if (nl < mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((ls.late[nl] >> i) & 1) d |= ls.in_block[i];
            d &= ls.anc[n0 + nl];
        }
        s.draft[nl] = d;
    }
    __syncthreads();
    const int U = s.total;
    const int page_tiles = (U + TPT - 1) / TPT;
    // tiles of this split (the first has tile 0, the drafted tokens; page tile i is tile i + 1)
    const int tiles = page_tiles + 1;
    const int t0 = (tiles * split + u.splits - 1) / u.splits, t1 = (tiles * (split + 1) + u.splits - 1) / u.splits;
    const int e_lo = max(0, t0 - 1) * TPT, e_hi = min(U, max(0, t1 - 1) * TPT);
#pragma unroll
    for (int x = 0; x < EPT; ++x) {
        if (id[x] < 0) continue;
        const int c = id[x], at = ls.before[c >> 5] + __popc(ls.bits[c >> 5] & ((1u << (c & 31)) - 1u));
        if (at < e_lo || at >= e_hi) continue;
        const int nl = list_of(tid + x * NT);
        atomicOr(reinterpret_cast<uint32_t*>(&s.mask[at - e_lo]) + (nl >> 5), 1u << (nl & 31));
        s.page[at - e_lo] = pg[x];
    }
    // keys of the last page tile: the cache's last page, if chosen, holds len % block_k
    const int last_keys = (U - (page_tiles - 1) * TPT) * BK - (s.partial ? BK - len % BK : 0);
    auto tile_keys = [&](int t) { return t == 0 ? nodes : t < page_tiles ? kTile : last_keys; };
    cp_async_wait_all();
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    const int n_tiles = t1 - t0;

    if (warp == kTmaWarp) {
        // -------------------------------------------------------------------- TMA producer
        const bool leader = elect_one();
        int j = 0;
        bool ok = true;
        for (; j < n_tiles; ++j) {
            const int t = t0 + j;
            if (t == 0) continue;  // under way since the start
            const int e0 = (t - 1) * TPT, cnt = min(TPT, U - e0);
            int rows[TPT];
#pragma unroll
            for (int x = 0; x < TPT; ++x) rows[x] = x < cnt ? s.page[e0 + x - e_lo] * BK : 0;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                uint64_t* fullb = kv ? &s.v_full : &s.k_full;
                if (ok && j > 0) ok = mbar_wait(kv ? &s.v_empty : &s.k_empty, (j - 1) & 1, a.status, 0xc11);
                if (!ok) break;
                if (leader) {
                    uint8_t* dst = kv ? s.v : s.k;
                    mbar_arrive_expect_tx(fullb, (uint32_t)cnt * BK * D * 2);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
#pragma unroll
                        for (int x = 0; x < TPT; ++x)
                            if (x < cnt)
                                tma_load_3d(dst + h * kHalf + x * BK * 128, kv ? &tm_vp : &tm_kp, fullb, 64 * h, r, rows[x]);
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        // no copy of ours may still be landing when the CTA leaves
        if (j > 0) {
            mbar_wait(&s.k_full, (j - 1) & 1, a.status, 0xc12);
            mbar_wait(&s.v_full, (j - 1) & 1, a.status, 0xc13);
        }
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------------------------- MMA issuer
        const bool leader = elect_one();
        const uint64_t dq = umma_sdesc(smem_u32(s.q), 16, 1024, 2), dk = umma_sdesc(smem_u32(s.k), 16, 1024, 2);
        const uint64_t dv = umma_sdesc(smem_u32(s.v), kHalf, 1024, 2);
        constexpr uint32_t kIdescO = umma_idesc_bf16(kRows, D, false, true);
        bool ok = true;
        for (int j = 0; ok && j <= n_tiles; ++j) {  // PV of tile j - 1, S of tile j
            if (j > 0) {
                const int steps = (tile_keys(t0 + j - 1) + 15) / 16;
                ok = mbar_wait(&s.v_full, (j - 1) & 1, a.status, 0xc23) && mbar_wait(&s.p_ready, (j - 1) & 1, a.status, 0xc24);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < kTile / 16; ++ks)  // P of keys 64 .. 127 starts at column 64
                        if (ks < steps)
                            umma_bf16_tmem_a(tmem + kColO, tmem + (ks / 4) * 64 + (ks & 3) * 8, dv + ((ks * 16 * 128) >> 4), kIdescO,
                                             j > 1 || ks > 0);
                    umma_commit(&s.v_empty);
                    if (j == n_tiles) umma_commit(&s.pv_done);
                }
                __syncwarp();
            }
            if (j < n_tiles) {
                ok = mbar_wait(&s.k_full, j & 1, a.status, 0xc22);
                if (!ok) break;
                tc_fence_after();
                const uint32_t idesc = umma_idesc_bf16(kRows, 0, false, false) | ((uint32_t)(tile_keys(t0 + j) + 15) / 16 << 18);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = ((ks / 4) * kHalf + (ks & 3) * 32) >> 4;
                        umma_bf16(tmem, dq + off, dk + off, idesc, ks > 0);
                    }
                    umma_commit(&s.s_full);
                    umma_commit(&s.k_empty);
                }
                __syncwarp();
            }
        }
        if (leader) umma_commit(&s.drain);
        mbar_wait(&s.drain, 0, a.status, 0xc25);
    } else {
        // -------------------------------------------------------------------- softmax: two threads per row
        // Thread (hf, row): columns 64 hf .. 64 hf + 63 of S.
        constexpr int CW = D / 2;  // output columns of a thread
        const int hf = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t pair_bar = 1 + (warp & 3);  // the two warps of these 32 rows
        const int nl = row >> lg;
        const bool live = nl < mine;
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lane_addr + hf * 64, tO = lane_addr + kColO + hf * CW;
        const float sl2 = a.scale * 1.4426950408889634f;
        const uint64_t sl2x2 = f2_packf(sl2, sl2);
        const uint32_t* my_mask = reinterpret_cast<const uint32_t*>(s.mask) + ((nl >> 5) & 1);  // this row's word of an entry
        const uint32_t my_bit = live ? 1u << (nl & 31) : 0u;
        float mref = -INFINITY;
        // the thread's part of the row's sum and of the sum of the weights as the product takes them, two halves each
        uint64_t l2 = f2_packf(0.f, 0.f), r2 = l2;
        bool ok = true;
        for (int j = 0; ok && j < n_tiles; ++j) {
            const int t = t0 + j, keys = tile_keys(t);
            const bool whole = t > 0 && keys == kTile;  // every column is a cached key
            // this thread's two chunks of 32 columns: all-ones or zero words; in a tile that is not whole the columns
            // one by one
            uint32_t see[2];
            if (t > 0) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int e = (t - 1) * TPT + (2 * hf + c) / (BK / 32);
                    see[c] = (TPT == 1 || e < U) && (my_mask[2 * (e - e_lo)] & my_bit) ? 0xffffffffu : 0u;
                    if (!whole) {
                        const int left = keys - 64 * hf - 32 * c;  // keys in this chunk
                        see[c] &= left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
                    }
                }
            } else {
                const unsigned long long d = live && hf == 0 ? s.draft[nl] : 0ull;
                see[0] = (uint32_t)d;
                see[1] = (uint32_t)(d >> 32);
            }
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&s.s_full, j & 1, a.status, 0xc32));
            // (this S was issued after the PV of the tile before: O is not being written)
            // rows of V behind the tile's last key, up to the product's depth, hold whatever the page or the
            // buffer held before: zeros, so that P = 0 there gives 0 even against NaN. (After the wait for S: before it, a warp
            // whose rows are masked could be a tile ahead, where V's barrier does not tell this tile from the one before.)
            const int pad = ((keys + 15) & ~15) - keys;
            if (ok && pad) {
                ok = __all_sync(0xffffffffu, mbar_wait(&s.v_full, j & 1, a.status, 0xc31));
                for (int i = hf * kRows + row; ok && i < pad * (D / 8); i += 2 * kRows) {
                    const int vr = keys + i / (D / 8), c = i % (D / 8);
                    *reinterpret_cast<uint4*>(s.v + (c / 8) * kHalf + swz(vr, (c % 8) * 16, 128)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
            }
            tc_fence_after();
            const bool any = ok && __any_sync(0xffffffffu, (see[0] | see[1]) != 0u);
            // S is read twice, 32 columns at a time: all 64 in registers spilled, and the reloads took longer than this
            float mx = -INFINITY;
            bool odd = false;  // a NaN or +inf among the scores
            if (any) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[32];
                    tmem_ld32(tS + 32 * c, x);
                    tmem_ld_wait();
                    reg_fence(x);
                    float* f = reinterpret_cast<float*>(x);
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = (see[c] >> e) & 1 ? f[e] : -INFINITY;
                    }
                    float m0 = max3n(f[0], f[1], f[2]), m1 = max3n(f[3], f[4], f[5]);
#pragma unroll
                    for (int e = 6; e < 30; e += 4) {
                        m0 = max3n(m0, f[e], f[e + 1]);
                        m1 = max3n(m1, f[e + 2], f[e + 3]);
                    }
                    m0 = max3n(m0, m1, max3n(f[30], f[31], f[31]));
                    const bool strange = !(m0 < INFINITY);
                    odd = odd || strange;
                    // a NaN or +inf score that the row sees makes the row NaN (-inf is a weight of zero)
                    if (strange && see[c]) l2 = r2 = f2_packf(NAN, NAN);
                    mx = see[c] ? fmaxf(mx, m0) : mx;
                }
                mx *= sl2;
            }
            // the running maximum, common to the row's two threads, is only touched when one of the 64 has to (or a
            // wait ran out: the two warps leave together)
            if (bar_red_or(pair_bar, 64, !ok || j == 0 || mx > mref + 8.f)) {
                s.row_max[hf][row] = mx;
                if (bar_red_or(pair_bar, 64, !ok)) {
                    ok = false;
                    break;
                }
                const float m2 = fmaxf(mx, s.row_max[hf ^ 1][row]);
                const bool up = j == 0 || m2 > mref + 8.f;
                if (j > 0) {
                    tc_fence_after();
                    const float f = up ? fast_exp2(mref - m2) : 1.f;
                    l2 = f2_mul(l2, f2_packf(f, f));
                    r2 = f2_mul(r2, f2_packf(f, f));
#pragma unroll
                    for (int c = 0; c < CW / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16(tO + 16 * c, o);
                        tmem_ld_wait();
                        reg_fence(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st16(tO + 16 * c, o);
                    }
                }
                if (up) mref = m2;
            }
            if (!any) {
                uint32_t z[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = 0u;
                tmem_st16(tS, z);
                tmem_st16(tS + 16, z);
            } else {
                const float base = mref == -INFINITY ? 0.f : mref;
                // Whole tiles: a chunk that the row does not see gets base = +inf, so that every finite score gives
                // exactly 0. Others, and tiles with a NaN or an infinite score (maybe of rows that do not see it): the
                // unseen columns become -inf one by one.
                auto weights = [&](auto plain_c) {
                    constexpr bool kPlain = decltype(plain_c)::value;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t x[32], pk[16];
                        tmem_ld32(tS + 32 * c, x);
                        tmem_ld_wait();
                        reg_fence(x);
                        if (!kPlain) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = (see[c] >> e) & 1 ? x[e] : 0xff800000u;
                        }
                        const float nb = kPlain && !see[c] ? -INFINITY : -base;
                        const uint64_t nb2 = f2_packf(nb, nb);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float e0, e1;
                            f2_unpack(f2_fma(f2_pack(x[2 * e], x[2 * e + 1]), sl2x2, nb2), e0, e1);
                            e0 = fast_exp2(e0);
                            e1 = fast_exp2(e1);
                            l2 = f2_add(l2, f2_packf(e0, e1));
                            pk[e] = pack_bf16x2(e0, e1);
                            r2 = f2_add(r2, f2_pack(pk[e] << 16, pk[e] & 0xffff0000u));
                        }
                        tmem_st16(tS + 16 * c, pk);
                    }
                };
                if (whole && !__any_sync(0xffffffffu, odd)) weights(std::true_type{});
                else weights(std::false_type{});
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.p_ready);
        }
        // -------------------------------------------------------------------- outputs
        // Through shared memory (K and V are no longer read: the last PV is done), so that a warp writes whole rows: 32 rows
        // of 16-byte pieces straight from the lanes took 4 us at the end of every CTA. Q stays, for rows that are evaluated
        // token by token (the output may be written over the queries).
        if (ok && n_tiles > 0) {
            bool done = false;
            for (int i = 0; i < 32 && !done; ++i) done = mbar_try_wait(&s.pv_done, 0);  // before the timed wait's loads
            ok = __all_sync(0xffffffffu, done || mbar_wait(&s.pv_done, 0, a.status, 0xc34));
            tc_fence_after();
        }
        float l0, l1, r0, r1;
        f2_unpack(l2, l0, l1);
        f2_unpack(r2, r0, r1);
        s.row_sum[hf][row] = r0 + r1;
        s.row_max[hf][row] = l0 + l1;  // (the other warp's last read of a maximum came before its part of the last P)
        bar_sync_named(pair_bar, 64);
        if (ok) {
            const float l = s.row_max[0][row] + s.row_max[1][row];
            const bool part = u.splits > 1;
            const bool has = l > 0.f || l != l;  // a NaN sum stays NaN
            const float inv = has ? 1.f / (s.row_sum[0][row] + s.row_sum[1][row]) : 0.f;
            const float lse = has ? (mref + log2f(l)) * 0.6931471805599453f : -INFINITY;
            // rows are consecutive heads of consecutive nodes: row i of the CTA is head i % G of node n0 + i / G
            auto out_row = [&](int i) {
                return ((int64_t)b * a.T + n0 + (i >> lg)) * a.H_q + (r << lg) + (i & ((1 << lg) - 1));
            };
            const bool write = hf == 0 && n0 + nl < a.T;
            float odd_out = 0.f;  // NaN once one of the thread's outputs is not finite
            if (hf == 0 && part && row < a.part_rows) a.lse_part[u.part * a.part_rows + row] = lse;
            if (write && !part && a.lse) a.lse[out_row(row)] = lse;
            if (!part || n_tiles > 0) {
                uint8_t* stage = s.k + warp * (32 * CW * 4);
                auto store = [&](auto half_c, auto* base, auto at) {  // row i goes to row at(i) of base
                    constexpr bool kHalfOut = decltype(half_c)::value;
                    constexpr int LP = (kHalfOut ? 1 : 2) + (CW == 64 ? 2 : 1), P = 1 << LP;  // 16-byte pieces of a row
                    constexpr int SW = P - 1 < 7 ? P - 1 : 7;
#pragma unroll
                    for (int c = 0; c < CW / 32; ++c) {
                        uint32_t o[32];
                        if (n_tiles > 0) {
                            tmem_ld32(tO + 32 * c, o);
                            tmem_ld_wait();
                            reg_fence(o);
                        }
                        float f[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = has ? __uint_as_float(o[e]) * inv : 0.f;
#pragma unroll
                        for (int e = 0; e < 32; ++e) odd_out = fmaf(f[e], 0.f, odd_out);
#pragma unroll
                        for (int e = 0; e < (kHalfOut ? 4 : 8); ++e) {
                            uint4 val;
                            if (kHalfOut)
                                val = make_uint4(pack_bf16x2(f[8 * e], f[8 * e + 1]), pack_bf16x2(f[8 * e + 2], f[8 * e + 3]),
                                                 pack_bf16x2(f[8 * e + 4], f[8 * e + 5]), pack_bf16x2(f[8 * e + 6], f[8 * e + 7]));
                            else
                                val = make_uint4(__float_as_uint(f[4 * e]), __float_as_uint(f[4 * e + 1]),
                                                 __float_as_uint(f[4 * e + 2]), __float_as_uint(f[4 * e + 3]));
                            *reinterpret_cast<uint4*>(stage + lane * P * 16 + (((c * (kHalfOut ? 4 : 8) + e) ^ (lane & SW)) << 4)) = val;
                        }
                    }
                    __syncwarp();
                    constexpr int RP = 32 / P;  // rows a pass of the warp writes
                    const int pc = lane & (P - 1);
#pragma unroll
                    for (int i = 0; i < 32 / RP; ++i) {
                        const int rr = i * RP + lane / P, ri = (warp & 3) * 32 + rr;
                        if (n0 + (ri >> lg) < a.T)
                            *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(base + at(ri) * D + hf * CW) + pc * 16) =
                                *reinterpret_cast<const uint4*>(stage + rr * P * 16 + ((pc ^ (rr & SW)) << 4));
                    }
                };
                if (part) store(std::false_type{}, a.o_part + (int64_t)u.part * a.part_rows * D, [](int i) { return i; });
                else if (a.out_bf16) store(std::true_type{}, a.out_bf16, out_row);
                else store(std::false_type{}, a.out, out_row);
                // Rows with an output that is not finite, though no logit is NaN or +inf, again token by token.
                __syncwarp();
                for (unsigned again = __ballot_sync(0xffffffffu, odd_out != odd_out && l == l); again; again &= again - 1) {
                    const int x = __ffs(again) - 1, ri = (warp & 3) * 32 + x;
                    const float lse2 = __shfl_sync(0xffffffffu, mref + log2f(l), x);
                    const int64_t to = (part ? (int64_t)u.part * a.part_rows + ri : out_row(ri)) * D;
                    tree_row_by_tokens<D, BK>(a, s, b, r, ri, hf, t0 == 0, e_lo, e_hi,
                                              s.partial && e_hi == U ? len % BK : BK, lse2,
                                              part ? a.o_part + to : a.out ? a.out + to : nullptr,
                                              part || a.out ? nullptr : a.out_bf16 + to);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 256);
    pdl_trigger();
}

// Items split over CTAs: log-sum-exp merge of their parts (at most 32), one warp per row (blockIdx.y: the item). A part
// that saw no token of the row has LSE = -inf and an output that is not read.
template <int D>
__global__ void __launch_bounds__(256) k_tree_combine(const __grid_constant__ TreeArgs a) {
    const int row = blockIdx.x * 8 + warp_id(), lane = threadIdx.x & 31, y = blockIdx.y;
    pdl_wait();
    const int2 count = *a.split_count;
    const int4 it = a.split_items[y];
    const int splits = count.y, step = count.x * a.part_rows, first = y * a.part_rows + row;  // the row in part p: first + p * step
    if (splits == 1 || y >= count.x || row >= a.part_rows) return;
    const float my_l = lane < splits ? a.lse_part[first + lane * step] : -INFINITY;
    const int node = it.z * (kRows >> a.lg_g) + (row >> a.lg_g);
    if (node >= a.T) return;
    const int64_t w = ((int64_t)it.x * a.T + node) * a.H_q + (it.y << a.lg_g) + (row & ((1 << a.lg_g) - 1));
    float mx = my_l;
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // Of a part that saw no token the weight is -1 here: its output may never have been written, and is dropped. That of
    // one whose weight underflows to 0 is not: an infinity or NaN there makes the row NaN, as it does within a part.
    const float my_w = my_l == -INFINITY ? -1.f : __expf(my_l - mx);
    float z = my_l == -INFINITY ? 0.f : my_w;
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    constexpr int kPer = D / 32;
    float acc[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) acc[x] = 0.f;
    // Six parts under way at a time, without branches (one by one the 18 parts of a single node took 4 us longer).
    for (int p0 = 0; p0 < splits; p0 += 6) {
        float f[6][kPer], wp[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            const int p = min(p0 + i, splits - 1);
            wp[i] = __shfl_sync(0xffffffffu, my_w, p);
            if (p0 + i >= splits) wp[i] = -1.f;
            const float* o = a.o_part + (int64_t)(first + p * step) * D + lane * kPer;
            if (kPer == 4) {
                const float4 v = *reinterpret_cast<const float4*>(o);
                f[i][0] = v.x, f[i][1] = v.y, f[i][kPer - 2] = v.z, f[i][kPer - 1] = v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2*>(o);
                f[i][0] = v.x, f[i][1] = v.y;
            }
        }
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
            for (int x = 0; x < kPer; ++x) acc[x] = wp[i] < 0.f ? acc[x] : fmaf(wp[i], f[i][x], acc[x]);
    }
    const float inv = z > 0.f || z != z ? 1.f / z : 0.f;
    if (a.out_bf16) {
        __nv_bfloat16* o = a.out_bf16 + w * D + lane * kPer;
#pragma unroll
        for (int x = 0; x < kPer; x += 2)
            *reinterpret_cast<uint32_t*>(o + x) = pack_bf16x2(acc[x] * inv, acc[x + 1] * inv);
    } else {
        float* o = a.out + w * D + lane * kPer;
#pragma unroll
        for (int x = 0; x < kPer; ++x) o[x] = acc[x] * inv;
    }
    if (lane == 0 && a.lse) a.lse[w] = z == 0.f ? -INFINITY : mx + logf(z);
}

int tree_ctas(int B, int T, int H_q, int H_kv) {
    const int per = kRows / (H_q / H_kv);  // nodes per CTA
    return B * H_kv * ((T + per - 1) / per);
}

}  // namespace

// (at most one split per tile of a single node's list)
void tree_attn_plan(TreeArgs* a, int num_sms) {
    const int tpt = kTile / a->block_k;
    a->slots = 2 * num_sms;
    a->max_splits = std::min((a->topk + tpt) / tpt + 1, 32);
    a->part_rows = std::min(kRows, a->T * (a->H_q / a->H_kv));
}
// Partial outputs that may be under way: of `slots` CTAs, or fewer where there are few items.
static size_t tree_parts(const TreeArgs& a) {
    return std::min<size_t>(a.slots, (size_t)tree_ctas(a.B, a.T, a.H_q, a.H_kv) * a.max_splits);
}
size_t tree_attn_ws_bytes(const TreeArgs& a) {
    return ((tree_parts(a) * a.part_rows * (a.d + 1) * 4 + 15) & ~size_t(15)) + (a.slots / 2) * sizeof(int4) + 16;
}
void tree_attn_carve(TreeArgs* a, void* base) {
    a->o_part = static_cast<float*>(base);
    const size_t rows = tree_parts(*a) * a->part_rows;
    a->lse_part = a->o_part + rows * a->d;
    a->split_items = reinterpret_cast<int4*>(static_cast<uint8_t*>(base) + ((rows * (a->d + 1) * 4 + 15) & ~size_t(15)));
    a->split_count = reinterpret_cast<int2*>(a->split_items + a->slots / 2);
}

cudaError_t run_tree_attn(const TreeArgs& a, const void* q, const void* k, const void* v, const void* k_pool,
                          const void* v_pool, cudaStream_t st) {
    CUtensorMap kp, vp, kd, vd;
    const uint64_t es = 2, row = (uint64_t)a.H_kv * a.d * es;
    const uint64_t dims[4] = {(uint64_t)a.d, (uint64_t)a.H_kv, (uint64_t)a.T, (uint64_t)a.B};
    const uint64_t strides[3] = {(uint64_t)a.d * es, row, row * a.T};
    const uint32_t box[4] = {64, 1, 64, 1};
    const uint64_t slots = (uint64_t)a.num_pages * a.block_k;
    if (!make_tmap_3d(&kp, k_pool, a.d, a.H_kv, slots, a.d * es, row, 64, 1, a.block_k, 128) ||
        !make_tmap_3d(&vp, v_pool, a.d, a.H_kv, slots, a.d * es, row, 64, 1, a.block_k, 128) ||
        !make_tmap_4d(&kd, k, dims, strides, box, 128) || !make_tmap_4d(&vd, v, dims, strides, box, 128))
        return cudaErrorInvalidValue;
    const int items = tree_ctas(a.B, a.T, a.H_q, a.H_kv), parts = (int)tree_parts(a);
    const dim3 grid(items / a.slots * a.slots + (items % a.slots ? parts : 0));  // enough for any number of live items
    const auto* qb = static_cast<const __nv_bfloat16*>(q);
    TreeArgs args = a;
    args.k = static_cast<const __nv_bfloat16*>(k), args.v = static_cast<const __nv_bfloat16*>(v);
    args.k_pool = static_cast<const __nv_bfloat16*>(k_pool), args.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
    auto pick = [&](auto d_c, auto bk_c) -> cudaError_t {
        constexpr int D = decltype(d_c)::value, BK = decltype(bk_c)::value;
        const size_t smem = std::max<size_t>(sizeof(TreeAttnSmem<D>) + 1024, 100 * 1024);  // at most two CTAs an SM
        auto kern = k_tree_attn<D, BK>;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        kern<<<grid, kAttnThreads, smem, st>>>(kp, vp, kd, vd, args, qb);
        return cudaGetLastError();
    };
    using I32 = std::integral_constant<int, 32>;
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    cudaError_t e;
    {
        ProfScope ps("tree_attn", st);
        if (a.d == 128)
            e = a.block_k == 128 ? pick(I128{}, I128{}) : a.block_k == 64 ? pick(I128{}, I64{}) : pick(I128{}, I32{});
        else
            e = a.block_k == 128 ? pick(I64{}, I128{}) : a.block_k == 64 ? pick(I64{}, I64{}) : pick(I64{}, I32{});
    }
    if (e != cudaSuccess) return e;
    ProfScope ps("tree_combine", st);
    const dim3 cgrid((a.part_rows + 7) / 8, std::min(items, a.slots / 2));
    return a.d == 128 ? launch_pdl(k_tree_combine<128>, cgrid, dim3(256), 0, st, a)
                      : launch_pdl(k_tree_combine<64>, cgrid, dim3(256), 0, st, a);
}

}  // namespace msa
