// Sparse attention of drafted-token trees over a paged cache. Row (node, head h of group r) attends the
// tokens of its virtual sequence (the cache, its ancestors, itself) that lie in the blocks of its list
// blocks[b, node, r, :]: softmax(q . k * scale) v.
//
// Query-outer: one CTA holds 128 NWG rows (128 NWG / G nodes with the G heads of one group) and walks the
// union of their selected pages, so that a page that several nodes chose, which is the rule (their queries
// are near), is loaded once per CTA and no partial outputs are spilled; a node that did not choose a page is
// masked there. The union is a bitmap over the sequence's blocks in shared memory, its order the block order,
// each entry with the set of nodes that chose it. Keys go in tiles of 128 (128 / block_k pages); the last
// tile is the drafted tokens, masked to each node's ancestors in its selected blocks.
//
// Per tile and warpgroup: S = Q K^T (tcgen05, M = N = 128) in TMEM; a thread owns one row, takes the tile's
// maximum, exponentials (base 2) and sums in fp32, writes P as bf16 over S; O += P V accumulates in TMEM.
// The running maximum is only raised, and O rescaled, when a row's maximum grows by more than 2^8: exponents
// stay far inside fp32 and bf16, and most tiles rescale nothing. O is normalised by the sum of the rounded P
// that the product used, the LSE by the exact sum, as in the prefill and decode kernels. bf16 P costs at most
// 2^-8 of each weight; the products and sums are fp32.
//
// NWG = 2 (more than 128 rows): two row tiles share K and V and alternate between the tensor cores and the
// exponentials. NWG = 1: two S buffers, so that the next tile's S runs under this tile's softmax. Where the
// CTAs do not fill the device the union is split over `splits` CTAs and merged by k_tree_combine.
#include "msa_tree.cuh"

namespace msa {

namespace {

constexpr int kRows = 128;
constexpr int kMaxEntries = kTreeMaxT * 17;  // union of a CTA's lists
constexpr int kWords = kTreeMaxBlocks / 32;

template <int D, int NWG>
struct TreeAttnSmem {
    alignas(1024) uint8_t q[NWG][kRows * D * 2];
    alignas(1024) uint8_t k[2][kTile * D * 2];
    alignas(1024) uint8_t v[2][kTile * D * 2];
    unsigned long long mask[kMaxEntries];   // nodes of the CTA that chose the entry
    unsigned long long anc[64], draft[64];  // ancestors of a node; drafted tokens that a node attends
    int page[kMaxEntries];
    int up[64];
    uint32_t late[64];                      // blocks >= len / block_k in a node's list
    uint32_t bits[kWords];
    int before[kWords];
    // s_full and p_ready: one per S buffer. A warp whose rows are masked runs ahead of the others, by one tile at
    // most, and must not arrive twice on one barrier for them.
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2], pv_done[2], drain;
    int total, last_partial;
    uint32_t tmem_base;
};

template <int D, int BK, int NWG>
__global__ void __launch_bounds__((4 * NWG + 2) * 32, 1)
    k_tree_attn(const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                const __grid_constant__ CUtensorMap tm_kd, const __grid_constant__ CUtensorMap tm_vd,
                const __grid_constant__ TreeArgs a, const __nv_bfloat16* __restrict__ q) {
    using Sm = TreeAttnSmem<D, NWG>;
    constexpr int TPT = kTile / BK;
    constexpr int NT = (4 * NWG + 2) * 32;
    constexpr uint32_t kHalf = kTile * 128;  // bytes of a 64-column half of a 128-row tile
    constexpr int kColO = 256;
    extern __shared__ uint8_t tree_raw[];
    Sm& s = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(tree_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
    const int G = a.H_q / a.H_kv, K1 = a.topk + 1;
    const int per_cta = NWG * kRows / G;  // nodes
    const int n_ct = (a.T + per_cta - 1) / per_cta;
    const int ct = blockIdx.x % n_ct, br = blockIdx.x / n_ct, r = br % a.H_kv, b = br / a.H_kv;
    const int split = blockIdx.y, n0 = ct * per_cta;
    const int len = tree_len(a, b), nodes = tree_nodes(a, b);
    const int full = len / BK, npages = (len + BK - 1) / BK;  // complete pages, pages
    const int64_t n_rows = (int64_t)a.B * a.T * a.H_q;
    if (tid == 0 && r == 0 && ct == 0 && split == 0 && (len != a.cache_len[b] || nodes != a.n_nodes[b]))
        raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xc01);

    // ------------------------------------------------------------------ the union of the CTA's lists
    if (tid < 64) tree_ancestors(a, b, nodes, s.anc, s.up, 1, 0xc02);
    for (int i = tid; i < kWords; i += NT) s.bits[i] = 0u;
    for (int i = tid; i < kMaxEntries; i += NT) s.mask[i] = 0ull;
    if (tid < 64) s.late[tid] = 0u;
    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s.k_full[x], 1);
            mbar_init(&s.k_empty[x], 1);
            mbar_init(&s.v_full[x], 1);
            mbar_init(&s.v_empty[x], 1);
            mbar_init(&s.s_full[x], 1);
            mbar_init(&s.p_ready[x], 4);
            mbar_init(&s.pv_done[x], 1);
        }
        mbar_init(&s.drain, 1);
        fence_mbar_init();
    }
    // Q rows (zero where the node does not exist), swizzled halves of 64 columns
    for (int i = tid; i < NWG * kRows * (D / 8); i += NT) {
        const int row = i / (D / 8), c = i % (D / 8), node = n0 + row / G, h = row % G;
        const uint32_t dst = smem_u32(s.q[0]) + (row / kRows) * (kRows * D * 2) + (c / 8) * kHalf +
                             swz(row % kRows, (c % 8) * 16, 128);
        const bool live = node < nodes;
        cp_async_16_zfill(dst, live ? q + (((int64_t)b * a.T + node) * a.H_q + r * G + h) * D + c * 8 : q, live);
    }
    if (warp == 4 * NWG + 1) {
        tmem_alloc(&s.tmem_base, 512);
        tmem_relinquish();
    }
    __syncthreads();
    const int mine = max(0, min(per_cta, nodes - n0));  // nodes of this CTA that exist
    for (int e = tid; e < mine * K1; e += NT) {
        const int nl = e / K1, n = n0 + nl;
        const int c = a.blocks[(((int64_t)b * a.T + n) * a.H_kv + r) * K1 + e % K1];
        if (c == -1) continue;
        if (c < -1 || c > (len + __popcll(s.anc[n]) - 1) / BK) {
            raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xc03);
            continue;
        }
        if (c < npages) atomicOr(&s.bits[c >> 5], 1u << (c & 31));
        if (c >= full) atomicOr(&s.late[nl], 1u << (c - full));
    }
    __syncthreads();
    if (warp == 0) {
        int sum = 0;
#pragma unroll
        for (int x = 0; x < kWords / 32; ++x) sum += __popc(s.bits[lane * (kWords / 32) + x]);
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        int at = incl - sum;
#pragma unroll
        for (int x = 0; x < kWords / 32; ++x) {
            s.before[lane * (kWords / 32) + x] = at;
            at += __popc(s.bits[lane * (kWords / 32) + x]);
        }
        if (lane == 31) s.total = incl;
        if (lane == 0) s.last_partial = npages > full && ((s.bits[full >> 5] >> (full & 31)) & 1);
    }
    if (tid >= 64 && tid - 64 < mine) {
        // drafted tokens that node n0 + tid - 64 attends: its ancestors in its selected blocks
        const int nl = tid - 64;
        unsigned long long left = s.anc[n0 + nl], d = 0ull;
        const uint32_t late = s.late[nl];
        while (left) {
            const int m = __ffsll(left) - 1;
            left &= left - 1;
            const int c = (len + __popcll(s.anc[m]) - 1) / BK;
            if ((late >> (c - full)) & 1) d |= 1ull << m;
        }
        s.draft[nl] = d;
    }
    __syncthreads();
    const int U = s.total;
    const int page_tiles = (U + TPT - 1) / TPT;
    // tiles of this split: page tiles, then the drafted tokens' tile; none where the CTA has no nodes
    const int tiles = mine > 0 ? page_tiles + 1 : 0;
    const int t0 = (int)((int64_t)tiles * split / a.splits), t1 = (int)((int64_t)tiles * (split + 1) / a.splits);
    const int e_lo = t0 * TPT, e_hi = min(U, t1 * TPT);
    for (int e = tid; e < mine * K1; e += NT) {
        const int nl = e / K1, n = n0 + nl;
        const int c = a.blocks[(((int64_t)b * a.T + n) * a.H_kv + r) * K1 + e % K1];
        if (c < 0 || c >= npages || c > (len + __popcll(s.anc[n]) - 1) / BK) continue;
        const int x = s.before[c >> 5] + __popc(s.bits[c >> 5] & ((1u << (c & 31)) - 1u));
        if (x < e_lo || x >= e_hi) continue;
        atomicOr(&s.mask[x - e_lo], 1ull << nl);
        s.page[x - e_lo] = tree_page(a, b, c, 0xc04);
    }
    cp_async_wait_all();
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    const int n_tiles = t1 - t0;
    // keys of local tile j: pages hold block_k each, the cache's last page len % block_k, the last tile the nodes
    auto tile_keys = [&](int j) {
        const int t = t0 + j;
        if (t == page_tiles) return nodes;
        const int cnt = min(TPT, U - t * TPT);
        return t == page_tiles - 1 && s.last_partial ? (cnt - 1) * BK + len % BK : cnt * BK;
    };

    if (warp == 4 * NWG) {
        // -------------------------------------------------------------------- TMA producer
        if (lane == 0) {
            int j = 0;
            bool ok = true;
            for (; j < n_tiles; ++j) {
                const int st = j & 1, t = t0 + j;
                const bool drafted = t == page_tiles;
                const int cnt = drafted ? 1 : min(TPT, U - t * TPT);
                const uint32_t bytes = drafted ? 64u * D * 2 : (uint32_t)cnt * BK * D * 2;
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    uint64_t* fullb = kv ? &s.v_full[st] : &s.k_full[st];
                    if (j >= 2 && !mbar_wait(kv ? &s.v_empty[st] : &s.k_empty[st], ((j >> 1) - 1) & 1, a.status, 0xc11)) {
                        ok = false;
                        break;
                    }
                    uint8_t* dst = kv ? s.v[st] : s.k[st];
                    mbar_arrive_expect_tx(fullb, bytes);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        if (drafted)
                            tma_load_4d(dst + h * kHalf, kv ? &tm_vd : &tm_kd, fullb, 64 * h, r, 0, b);
                        else
                            for (int x = 0; x < cnt; ++x)
                                tma_load_3d(dst + h * kHalf + x * BK * 128, kv ? &tm_vp : &tm_kp, fullb, 64 * h, r,
                                            s.page[t * TPT + x - e_lo] * BK);
                    }
                }
                if (!ok) break;
            }
            // no copy of ours may still be landing when the CTA leaves
            for (int m = max(0, j - 2); m < j; ++m) {
                mbar_wait(&s.k_full[m & 1], (m >> 1) & 1, a.status, 0xc12);
                mbar_wait(&s.v_full[m & 1], (m >> 1) & 1, a.status, 0xc13);
            }
        }
    } else if (warp == 4 * NWG + 1) {
        // -------------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            auto issue_s = [&](int w, int j) {
                const uint32_t nk = (uint32_t)(tile_keys(j) + 15) & ~15u;
                const uint32_t idesc = umma_idesc_bf16(kRows, 0, false, false) | ((nk >> 3) << 17);
                const uint32_t qb = smem_u32(s.q[w]), kb = smem_u32(s.k[j & 1]);
                const int buf = NWG == 1 ? (j & 1) : w;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = (ks / 4) * kHalf + (ks & 3) * 32;
                    umma_bf16(tmem + buf * kTile, umma_sdesc(qb + off, 16, 1024, 2), umma_sdesc(kb + off, 16, 1024, 2),
                              idesc, ks > 0);
                }
                umma_commit(&s.s_full[buf]);
                if (w == NWG - 1) umma_commit(&s.k_empty[j & 1]);
            };
            constexpr uint32_t kIdescO = umma_idesc_bf16(kRows, D, false, true);
            bool ok = true;
            if (n_tiles > 0) {
                ok = mbar_wait(&s.k_full[0], 0, a.status, 0xc21);
                tc_fence_after();
                for (int w = 0; ok && w < NWG; ++w) issue_s(w, 0);
            }
            for (int j = 0; ok && j < n_tiles; ++j) {
                const bool more = j + 1 < n_tiles;
                if (more) ok = mbar_wait(&s.k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, a.status, 0xc22);
                if (NWG == 1 && ok && more) {
                    tc_fence_after();
                    issue_s(0, j + 1);
                }
                ok = ok && mbar_wait(&s.v_full[j & 1], (j >> 1) & 1, a.status, 0xc23);
                const int steps = (tile_keys(j) + 15) / 16;
                for (int w = 0; ok && w < NWG; ++w) {
                    ok = mbar_wait(&s.p_ready[NWG == 1 ? (j & 1) : w], (NWG == 1 ? j >> 1 : j) & 1, a.status, 0xc24);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t tP = tmem + (NWG == 1 ? (j & 1) : w) * kTile, vb = smem_u32(s.v[j & 1]);
                    for (int ks = 0; ks < steps; ++ks)
                        umma_bf16_tmem_a(tmem + kColO + w * kRows, tP + 8 * ks, umma_sdesc(vb + ks * 16 * 128, kHalf, 1024, 2),
                                         kIdescO, j > 0 || ks > 0);
                    umma_commit(&s.pv_done[w]);
                    if (w == NWG - 1) umma_commit(&s.v_empty[j & 1]);
                    if (NWG == 2 && more) issue_s(w, j + 1);
                }
            }
            umma_commit(&s.drain);
            mbar_wait(&s.drain, 0, a.status, 0xc25);
        }
    } else {
        // -------------------------------------------------------------------- softmax: one row per thread
        const int w = warp >> 2, row = (warp & 3) * 32 + lane;
        const int nl = (w * kRows + row) / G, h = (w * kRows + row) % G;
        const bool live = nl < mine;
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tO = lane_addr + kColO + w * kRows;
        const float sl2 = a.scale * 1.4426950408889634f;
        const unsigned long long draft = live ? s.draft[nl] : 0ull;
        float mref = -INFINITY, l = 0.f, lr = 0.f;
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
            const int t = t0 + j, keys = tile_keys(j), buf = NWG == 1 ? (j & 1) : w;
            // columns of each 32-column chunk that this row sees
            uint32_t see[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (t == page_tiles) {
                    see[c] = c < 2 ? (uint32_t)(draft >> (32 * c)) : 0u;
                } else {
                    const int left = keys - 32 * c;  // keys in this chunk
                    const uint32_t there = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
                    const int e = t * TPT + c / (BK / 32) - e_lo;
                    see[c] = live && left > 0 && ((s.mask[e] >> nl) & 1) ? there : 0u;
                }
            }
            // rows of V behind the tile's last key, up to the product's depth, hold whatever the page or the
            // stage held before: zeros, so that P = 0 there gives 0 even against NaN
            const int pad = ((keys + 15) & ~15) - keys;
            if (w == 0 && pad) {
                if (!__all_sync(0xffffffffu, mbar_wait(&s.v_full[j & 1], (j >> 1) & 1, a.status, 0xc31))) ok = false;
                for (int i = row; ok && i < pad * (D / 8); i += kRows) {
                    const int vr = keys + i / (D / 8), c = i % (D / 8);
                    *reinterpret_cast<uint4*>(s.v[j & 1] + (c / 8) * kHalf + swz(vr, (c % 8) * 16, 128)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
            }
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&s.s_full[buf], (NWG == 1 ? j >> 1 : j) & 1, a.status, 0xc32));
            if (!ok) break;
            tc_fence_after();
            const uint32_t tS = lane_addr + buf * kTile;
            const bool any = __any_sync(0xffffffffu, (see[0] | see[1] | see[2] | see[3]) != 0u);
            if (!any) {
                uint32_t z[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = 0u;
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_st16(tS + 16 * c, z);
            } else {
                uint32_t x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, x[c]);
                tmem_ld_wait();
                const bool whole = __all_sync(0xffffffffu, (see[0] & see[1] & see[2] & see[3]) == 0xffffffffu);
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    reg_fence(x[c]);
                    float* f = reinterpret_cast<float*>(x[c]);
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = (see[c] >> e) & 1 ? f[e] : -INFINITY;
                    }
                    float m0 = max3f(f[0], f[1], f[2]), m1 = max3f(f[3], f[4], f[5]);
#pragma unroll
                    for (int e = 6; e < 30; e += 4) {
                        m0 = max3f(m0, f[e], f[e + 1]);
                        m1 = max3f(m1, f[e + 2], f[e + 3]);
                    }
                    mx = fmaxf(mx, max3f(m0, m1, fmaxf(f[30], f[31])));
                }
                mx *= sl2;
                if (j == 0) {
                    mref = mx;
                } else {
                    const bool up = mx > mref + 8.f;
                    if (__any_sync(0xffffffffu, up)) {
                        ok = __all_sync(0xffffffffu, mbar_wait(&s.pv_done[w], (j - 1) & 1, a.status, 0xc33));
                        if (!ok) break;
                        tc_fence_after();
                        const float f = up ? fast_exp2(mref - mx) : 1.f;
                        if (up) mref = mx;
                        l *= f;
                        lr *= f;
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(tO + 16 * c, o);
                            tmem_ld_wait();
                            reg_fence(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(tO + 16 * c, o);
                        }
                    }
                }
                const float base = mref == -INFINITY ? 0.f : mref;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float* f = reinterpret_cast<const float*>(x[c]);
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float p0 = fast_exp2(fmaf(f[2 * e], sl2, -base)), p1 = fast_exp2(fmaf(f[2 * e + 1], sl2, -base));
                        l += p0 + p1;
                        pk[e] = pack_bf16x2(p0, p1);
                        lr += __uint_as_float(pk[e] << 16) + __uint_as_float(pk[e] & 0xffff0000u);
                    }
                    tmem_st16(tS + 16 * c, pk);
                }
            }
            tmem_st_wait();
            // every phase of pv_done is waited for in turn (a parity wait cannot tell a phase from the next but
            // one): PV of the previous tile ran under this tile's exponentials, so this costs nothing
            if (j > 0) ok = __all_sync(0xffffffffu, mbar_wait(&s.pv_done[w], (j - 1) & 1, a.status, 0xc35));
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.p_ready[buf]);
        }
        // -------------------------------------------------------------------- outputs
        if (ok && n_tiles > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&s.pv_done[w], (n_tiles - 1) & 1, a.status, 0xc34));
            tc_fence_after();
        }
        const int node = n0 + nl;
        if (ok) {
            const int64_t orow = ((int64_t)b * a.T + node) * a.H_q + r * G + h;
            const bool write = node < a.T, has = l > 0.f || l != l;  // a NaN sum stays NaN
            const float inv = has ? 1.f / lr : 0.f;
            const float lse = has ? (mref + log2f(l)) * 0.6931471805599453f : -INFINITY;
            const bool part = a.splits > 1;
            if (write && part) a.lse_part[split * n_rows + orow] = lse;
            if (write && !part && a.lse) a.lse[orow] = lse;
            if (!part || n_tiles > 0) {
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16];
                    if (n_tiles > 0) {
                        tmem_ld16(tO + 16 * c, o);
                        tmem_ld_wait();
                        reg_fence(o);
                    }
                    float f[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = has ? __uint_as_float(o[e]) * inv : 0.f;
                    if (!write) continue;
                    if (!part && a.out_bf16) {
                        uint4* dst = reinterpret_cast<uint4*>(a.out_bf16 + orow * D + 16 * c);
                        dst[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
                        dst[1] = make_uint4(pack_bf16x2(f[8], f[9]), pack_bf16x2(f[10], f[11]), pack_bf16x2(f[12], f[13]), pack_bf16x2(f[14], f[15]));
                    } else {
                        float4* dst = reinterpret_cast<float4*>((part ? a.o_part + split * n_rows * D : a.out) + orow * D + 16 * c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) dst[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4 * NWG + 1) tmem_dealloc(tmem, 512);
    pdl_trigger();
}

// One warp per (node, head): log-sum-exp merge of the splits' partials (at most 32). A split that saw no
// token of the row has LSE = -inf and an output that is not read.
template <int D>
__global__ void __launch_bounds__(256) k_tree_combine(const __grid_constant__ TreeArgs a) {
    const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t n_rows = (int64_t)a.B * a.T * a.H_q;
    if (w >= n_rows) return;
    pdl_wait();
    const float my_l = lane < a.splits ? a.lse_part[lane * n_rows + w] : -INFINITY;
    float mx = my_l;
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float my_w = my_l == -INFINITY ? 0.f : __expf(my_l - mx);
    float z = my_w;
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    constexpr int kPer = D / 32;
    float acc[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) acc[x] = 0.f;
    for (int p = 0; p < a.splits; ++p) {
        const float wp = __shfl_sync(0xffffffffu, my_w, p);
        if (wp == 0.f) continue;
        const float* o = a.o_part + (p * n_rows + w) * D + lane * kPer;
#pragma unroll
        for (int x = 0; x < kPer; ++x) acc[x] = fmaf(wp, o[x], acc[x]);
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

// row tiles of 128 (node, head) rows that one CTA holds
int tree_wg(int T, int G) { return T * G > kRows ? 2 : 1; }
int tree_ctas(int B, int T, int H_q, int H_kv) {
    const int G = H_q / H_kv, per = tree_wg(T, G) * kRows / G;
    return B * H_kv * ((T + per - 1) / per);
}

}  // namespace

// Splits of the key walk: none once the CTAs fill the device; else as many as fill it, at most one per tile
// of a single node's list.
int tree_attn_splits(int B, int T, int H_q, int H_kv, int block_k, int topk, int num_sms) {
    const int tpt = kTile / block_k, tiles = (topk + 1 + tpt - 1) / tpt + 1;
    return std::max(1, std::min({tiles, num_sms / tree_ctas(B, T, H_q, H_kv), 32}));
}
size_t tree_attn_ws_bytes(int B, int T, int H_q, int d, int splits) {
    if (splits <= 1) return 0;
    const size_t rows = (size_t)splits * B * T * H_q;
    return ((rows * 4 + 255) & ~size_t(255)) + rows * d * 4;
}

cudaError_t run_tree_attn(const TreeArgs& a, const void* q, const void* k, const void* v, const void* k_pool,
                          const void* v_pool, cudaStream_t st) {
    const int G = a.H_q / a.H_kv;
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
    const int wg = tree_wg(a.T, G);
    const dim3 grid(tree_ctas(a.B, a.T, a.H_q, a.H_kv), a.splits);
    const auto* qb = static_cast<const __nv_bfloat16*>(q);
    auto launch = [&](auto kern, size_t bytes) -> cudaError_t {
        const size_t smem = std::max<size_t>(bytes + 1024, 120 * 1024);  // one CTA (512 TMEM columns) per SM
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        kern<<<grid, (4 * wg + 2) * 32, smem, st>>>(kp, vp, kd, vd, a, qb);
        return cudaGetLastError();
    };
    auto pick = [&](auto d_c, auto bk_c) -> cudaError_t {
        constexpr int D = decltype(d_c)::value, BK = decltype(bk_c)::value;
        return wg == 2 ? launch(k_tree_attn<D, BK, 2>, sizeof(TreeAttnSmem<D, 2>))
                       : launch(k_tree_attn<D, BK, 1>, sizeof(TreeAttnSmem<D, 1>));
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
    if (e != cudaSuccess || a.splits == 1) return e;
    ProfScope ps("tree_combine", st);
    const int64_t rows = (int64_t)a.B * a.T * a.H_q;
    const dim3 cgrid((unsigned)((rows + 7) / 8));
    return a.d == 128 ? launch_pdl(k_tree_combine<128>, cgrid, dim3(256), 0, st, a)
                      : launch_pdl(k_tree_combine<64>, cgrid, dim3(256), 0, st, a);
}

}  // namespace msa
