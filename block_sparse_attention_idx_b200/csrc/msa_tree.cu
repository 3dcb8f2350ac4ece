// Drafted-token trees over a paged cache: block selection for the T drafted tokens of each sequence
// (speculative decoding); msa_tree_attn.cu holds their attention. Node n of a tree, at depth e (its number of drafted ancestors),
// sits at position len + e and sees the len cached tokens, its ancestors and itself: its virtual sequence.
// Selection and attention are those of a decode step on that sequence, so that a drafted token gets the
// blocks and the output that it would get if its path had been decoded token by token.
//
// A page of the cache is one block. Blocks below len / block_k are whole pages; the virtual blocks from
// there on hold the cache's last tokens and the path's drafted tokens, whose K, V and K_idx are dense
// [B, T, ...] arrays: rejected tokens never reach the cache.
//
//   k_tree_scan    scores of all (node, group) rows of a sequence against every cached index key and their
//                  block maxima; ancestor sets
//   k_tree_topk    per (node, group): the drafted tokens' part of the last blocks, Top-k, local block
#include <algorithm>

#include "msa_tree.cuh"

namespace msa {

namespace {

// -------------------------------------------------------------------------------------- index scan
// Persistent CTAs (one per SM, a second grid dimension for every further 256 rows) take equal contiguous
// ranges of all sequences' 256-token tiles. S = Q_idx (128 (node, group) rows) . K_idx_tile^T on the tensor
// cores, so that one TMEM lane holds one row's scores and the block maxima need no exchange between lanes.
// Warps: 0-7 epilogue, 8 TMA, 9 MMA. Each warpgroup of the epilogue owns one of two 256-column accumulators:
// with more than 128 rows a row tile each, else alternate tiles. The sequence's Q_idx rows are staged twice, so
// that the next sequence's load overlaps this one's tiles.
// HBM-bound by design: each K_idx byte is read once for up to 256 rows. What else a tile costs is the issue of
// one warp (waits, descriptors, commits): some 1000 cycles, as long as the 16 KB of a 128-token tile take to
// arrive (1143 cycles a tile, 105 us for 16 sequences of up to 262144 tokens); hence tiles of 256 tokens and warp-uniform
// loops: 71 us for the same 407 MB, 0.87 of the copy rate, what the loads alone take.
constexpr int kScanThreads = 320;
constexpr int kScanTile = 256;

template <int DI>
struct TreeScanSmem {
    static constexpr int kStages = DI == 64 ? 4 : 8;
    alignas(1024) uint8_t q[2][2][kTile * DI * 2];
    alignas(1024) uint8_t k[kStages][kScanTile * DI * 2];
    uint64_t q_full[2], q_empty[2], k_full[kStages], k_empty[kStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base;
};

__device__ __forceinline__ int scan_tiles(const TreeArgs& a, int b) {
    return tree_nodes(a, b) > 0 ? (tree_len(a, b) + kScanTile - 1) / kScanTile : 0;
}
struct TileCursor {
    int b, tile, n, len;  // tile `tile` of sequence b, which has n tiles and len tokens
};
// Called by all lanes of a warp: the CTA's first tile and its number of tiles.
__device__ int tile_range(const TreeArgs& a, TileCursor& c) {
    const int lane = threadIdx.x & 31;
    long long T = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        int v = b0 + lane < a.B ? scan_tiles(a, b0 + lane) : 0;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        T += v;
    }
    const long long lo = T * blockIdx.x / gridDim.x, hi = T * (blockIdx.x + 1) / gridDim.x;
    long long cum = 0;
    for (int b0 = 0; b0 < a.B && lo < hi; b0 += 32) {
        const int v = b0 + lane < a.B ? scan_tiles(a, b0 + lane) : 0;
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, cum + incl > lo);
        if (hit) {
            const int l = __ffs(hit) - 1;
            c.b = b0 + l;
            c.n = __shfl_sync(0xffffffffu, v, l);
            c.tile = (int)(lo - (cum + __shfl_sync(0xffffffffu, incl, l) - c.n));
            c.len = tree_len(a, c.b);
            return (int)(hi - lo);
        }
        cum += __shfl_sync(0xffffffffu, incl, 31);
    }
    c.b = a.B;
    c.tile = c.n = c.len = 0;
    return 0;
}
// Moves to the next tile; true if it belongs to another sequence.
__device__ __forceinline__ bool tile_next(const TreeArgs& a, TileCursor& c) {
    if (++c.tile < c.n) return false;
    c.tile = 0;
    while (++c.b < a.B && (c.n = scan_tiles(a, c.b)) == 0) {}
    if (c.b < a.B) c.len = tree_len(a, c.b);
    return true;
}

template <int DI, int BK>
__global__ void __launch_bounds__(kScanThreads, 1)
    k_tree_scan(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ TreeArgs a) {
    using Sm = TreeScanSmem<DI>;
    constexpr int kStages = Sm::kStages;
    constexpr int TPT = kScanTile / BK;  // pages per tile
    constexpr uint32_t kPageBytes = BK * DI * 2, kTileBytes = kScanTile * DI * 2, kQBytes = kTile * DI * 2;
    constexpr uint32_t kLayout = DI == 64 ? 2u : 4u;
    constexpr uint32_t kSBO = 8 * DI * 2;
    constexpr uint32_t kIdesc = umma_idesc_bf16(kTile, kScanTile, false, false);
    extern __shared__ uint8_t tree_raw[];
    Sm& s = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(tree_raw) + 1023) & ~uintptr_t(1023));
    const int warp = warp_id(), lane = lane_id();
    const int R = a.T * a.H_kv;                             // (node, group) rows of a sequence
    const int row0 = blockIdx.y * 2 * kTile;
    const int rt = min(2, (R - row0 + kTile - 1) / kTile);  // row tiles of this CTA
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s.q_full[x], 1);
            mbar_init(&s.q_empty[x], 1);
            mbar_init(&s.acc_full[x], 1);
            mbar_init(&s.acc_empty[x], 4);
        }
        for (int x = 0; x < kStages; ++x) {
            mbar_init(&s.k_full[x], 1);
            mbar_init(&s.k_empty[x], 1);
        }
        mbar_init(&s.drain, 1);
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&s.tmem_base, 512);
        tmem_relinquish();
    }
    TileCursor cur;
    const int count = tile_range(a, cur);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;

    if (warp == 8) {
        // ------------------------------------------------------------------------ TMA producer
        const bool leader = elect_one();
        int n = 0, nq = -1, base = -32, page = 0;  // page: lane l holds the id of block base + l
        int st = 0;
        uint32_t ph = 1;  // parity that a stage's release has, before its first use the one that is already over
        bool fresh = true, ok = true;
        for (; n < count; ++n) {
            if (fresh) {
                ++nq;
                const int qs = nq & 1;
                ok = nq < 2 || mbar_wait(&s.q_empty[qs], ((nq >> 1) - 1) & 1, a.status, 0xb01);
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(&s.q_full[qs], (uint32_t)rt * kQBytes);
                    for (int x = 0; x < rt; ++x) tma_load_3d(s.q[qs][x], &tm_q, &s.q_full[qs], 0, row0 + x * kTile, cur.b);
                }
                __syncwarp();
                base = -32;
            }
            const int c0 = cur.tile * TPT;
            const int blocks = (cur.len + BK - 1) / BK;
            if (base < 0 || c0 >= base + 32) {  // TPT divides 32: a tile's pages never straddle a refill
                base = c0 & ~31;
                page = base + lane < blocks ? tree_page(a, cur.b, base + lane, 0xb02) : 0;
            }
            const int np = min(TPT, blocks - c0);
            ok = mbar_wait(&s.k_empty[st], ph, a.status, 0xb03);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (leader) mbar_arrive_expect_tx(&s.k_full[st], np * kPageBytes);
            __syncwarp();
#pragma unroll
            for (int x = 0; x < TPT; ++x) {
                const int p = __shfl_sync(0xffffffffu, page, (c0 + x) & 31);
                if (leader && x < np) tma_load_2d(s.k[st] + x * kPageBytes, &tm_k, &s.k_full[st], 0, p * BK);
            }
            __syncwarp();
            if (++st == kStages) {
                st = 0;
                ph ^= 1;
            }
            fresh = tile_next(a, cur);
        }
        // no copy of ours may still be landing when the CTA leaves
        for (int m = max(0, n - kStages); m < n; ++m)
            mbar_wait(&s.k_full[m % kStages], (m / kStages) & 1, a.status, 0xb04);
        for (int m = max(0, nq - 1); m <= nq; ++m)
            if (ok || m < nq) mbar_wait(&s.q_full[m & 1], (m >> 1) & 1, a.status, 0xb05);
    } else if (warp == 9) {
        // ------------------------------------------------------------------------ MMA issuer
        const bool leader = elect_one();
        const uint64_t dq = umma_sdesc(smem_u32(s.q[0][0]), 16, kSBO, kLayout), dk = umma_sdesc(smem_u32(s.k[0]), 16, kSBO, kLayout);
        int nq = -1, st = 0;
        uint32_t ph = 0;
        bool fresh = true, ok = true;
        for (int n = 0; ok && n < count; ++n) {
            if (fresh) {
                ++nq;
                ok = mbar_wait(&s.q_full[nq & 1], (nq >> 1) & 1, a.status, 0xb11);
            }
            ok = ok && mbar_wait(&s.k_full[st], ph, a.status, 0xb12);
            for (int x = 0; ok && x < rt; ++x) {
                // accumulator: the row tile's, or alternate ones; use u of it waits for the release of use u - 1
                const int acc = rt == 2 ? x : n & 1, u = rt == 2 ? n : n >> 1;
                ok = mbar_wait(&s.acc_empty[acc], (u & 1) ^ 1, a.status, 0xb13);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint64_t qd = dq + (((nq & 1) * 2 + x) * kQBytes >> 4), kd = dk + (st * kTileBytes >> 4);
#pragma unroll
                    for (int ks = 0; ks < DI / 16; ++ks)
                        umma_bf16(tmem + acc * kScanTile, qd + 2 * ks, kd + 2 * ks, kIdesc, ks > 0);
                    umma_commit(&s.acc_full[acc]);
                    if (x == rt - 1) umma_commit(&s.k_empty[st]);
                }
                __syncwarp();
            }
            if (++st == kStages) {
                st = 0;
                ph ^= 1;
            }
            fresh = tile_next(a, cur);
            if (fresh && leader) umma_commit(&s.q_empty[nq & 1]);
            __syncwarp();
        }
        if (leader) umma_commit(&s.drain);
        mbar_wait(&s.drain, 0, a.status, 0xb14);
    } else {
        // ------------------------------------------------------------------------ epilogue
        const int wg = warp >> 2;
        const uint32_t tacc = tmem + ((uint32_t)((warp & 3) * 32) << 16) + wg * kScanTile;
        const int row = row0 + (rt == 2 ? wg * kTile : 0) + (warp & 3) * 32 + lane;
        const int step = rt == 2 ? 1 : 2;  // tiles between this warpgroup's
        if (step == 2 && wg == 1 && count > 1) tile_next(a, cur);
        uint32_t ph = 0;
        for (int n = step == 2 ? wg : 0; n < count; n += step) {
            if (!__all_sync(0xffffffffu, mbar_wait(&s.acc_full[wg], ph, a.status, 0xb22))) break;
            ph ^= 1;
            tc_fence_after();
            float cmax[8];  // maxima of 32-column chunks
            if (row - lane < R) {
                const int left = cur.len - cur.tile * kScanTile;  // keys of the tile that exist
#pragma unroll
                for (int hf = 0; hf < 4; ++hf) {
                    uint32_t v[2][32];
#pragma unroll
                    for (int q = 0; q < 2; ++q) tmem_ld32(tacc + hf * 64 + q * 32, v[q]);
                    tmem_ld_wait();
                    if (hf == 3) {  // the accumulator is read: the next product may start
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s.acc_empty[wg]);
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        reg_fence(v[q]);
                        float* f = reinterpret_cast<float*>(v[q]);
                        if (left < kScanTile) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = hf * 64 + q * 32 + e < left ? f[e] : -INFINITY;
                        }
                        float m0 = max3f(f[0], f[1], f[2]), m1 = max3f(f[3], f[4], f[5]);
#pragma unroll
                        for (int e = 6; e < 30; e += 4) {
                            m0 = max3f(m0, f[e], f[e + 1]);
                            m1 = max3f(m1, f[e + 2], f[e + 3]);
                        }
                        cmax[hf * 2 + q] = fmaxf(max3f(m0, m1, fmaxf(f[30], f[31])), -INFINITY);  // all NaN: -inf
                    }
                }
                if (row < R) {
                    float* out = a.bmax + ((int64_t)cur.b * R + row) * a.bmax_ld + cur.tile * TPT;
                    if constexpr (TPT == 8) {
                        reinterpret_cast<float4*>(out)[0] = make_float4(cmax[0], cmax[1], cmax[2], cmax[3]);
                        reinterpret_cast<float4*>(out)[1] = make_float4(cmax[4], cmax[5], cmax[6], cmax[7]);
                    } else if constexpr (TPT == 4) {
                        *reinterpret_cast<float4*>(out) = make_float4(fmaxf(cmax[0], cmax[1]), fmaxf(cmax[2], cmax[3]),
                                                                      fmaxf(cmax[4], cmax[5]), fmaxf(cmax[6], cmax[7]));
                    } else {
                        *reinterpret_cast<float2*>(out) =
                            make_float2(fmaxf(fmaxf(cmax[0], cmax[1]), fmaxf(cmax[2], cmax[3])),
                                        fmaxf(fmaxf(cmax[4], cmax[5]), fmaxf(cmax[6], cmax[7])));
                    }
                }
            } else {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.acc_empty[wg]);
            }
            tile_next(a, cur);
            if (step == 2 && n + 2 < count) tile_next(a, cur);
        }
        // the ancestor sets of the Top-k kernel
        if (warp == 7 && blockIdx.y == 0)
            for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
                const int nodes = tree_nodes(a, b);
                unsigned long long anc[2];
                tree_ancestors(a, nodes, load_parent(a, b, lane), load_parent(a, b, lane + 32), anc, 0xb21);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (lane + 32 * x < nodes) a.anc[(int64_t)b * a.T + lane + 32 * x] = anc[x];
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512);
    pdl_trigger();
}

// ------------------------------------------------------------------------------------------ Top-k
// Key of a candidate: order-preserving bits of its maximum, then the complement of its id: unique, and the
// larger key ranks first (ties: the lower block).
__device__ __forceinline__ unsigned long long cand_key(float v, int c) {
    const uint32_t u = __float_as_uint(v + 0.f);  // -0 ranks as 0
    return ((unsigned long long)((u & 0x80000000u) ? ~u : (u | 0x80000000u)) << 32) | (0xffffffffu - (uint32_t)c);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

// WPR warps rank one (node, group) row, PL candidates a lane. The (k+1)-th largest of a warp's 32 lane maxima bounds
// its (k+1)-th largest candidate from below, so only the candidates at or above that bound, about 1.3 (k+1) of them
// and never more than k+1 lanes' worth, go to a list in shared memory, where each is ranked by counting. One pass
// over the maxima held in registers, no histogram, no sort. The list's worst case sizes the shared memory: with
// 64 candidates a lane for every row count, 2048 rows of 391 blocks took 17 us at 6 CTAs an SM.
constexpr int kTopkWarps = 4;

template <int WPR, int PL>
__global__ void __launch_bounds__(kTopkWarps * 32) k_tree_topk(const __grid_constant__ TreeArgs a, const __nv_bfloat16* __restrict__ q_idx,
                                                               const __nv_bfloat16* __restrict__ k_idx) {
    constexpr int RPC = kTopkWarps / WPR;  // rows per CTA
    constexpr int kPerLane = PL;           // candidates a lane can hold
    constexpr int kCap = 17 * PL + 4;      // survivors of a warp: at most topk + 1 lanes' candidates, and the last blocks
    __shared__ unsigned long long s_list[kTopkWarps * kCap];
    __shared__ int s_cnt[RPC], s_chosen[RPC][16];
    __shared__ uint32_t s_draft[RPC][4];
    __shared__ float s_kth[RPC][2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp / WPR, sub = warp % WPR;
    const int R = a.T * a.H_kv, K1 = a.topk + 1;
    const int64_t gr = (int64_t)blockIdx.x * RPC + slot;  // row of all sequences
    const bool live_row = gr < (int64_t)a.B * R;
    const int b = live_row ? (int)(gr / R) : 0, row = live_row ? (int)(gr % R) : 0;
    const int n = row / a.H_kv, g = row % a.H_kv;
    const int len = tree_len(a, b), nodes = tree_nodes(a, b);
    if (live_row && row == 0 && sub == 0 && lane == 0 && (len != a.cache_len[b] || nodes != a.n_nodes[b]))
        raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xb31);
    const bool live = live_row && n < nodes;
    pdl_wait();  // the maxima and the ancestor sets come from the scan
    // candidates 4 (lane + 32 sub) + 128 WPR j + {0..3}; loaded before it is known which of them exist
    const float* vals = a.bmax + ((int64_t)b * R + row) * a.bmax_ld;
    float v[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane / 4; ++j) {
        const int c = 4 * (lane + 32 * sub) + 128 * WPR * j;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && c < a.bmax_ld) f = *reinterpret_cast<const float4*>(vals + c);
        v[4 * j] = f.x;
        v[4 * j + 1] = f.y;
        v[4 * j + 2] = f.z;
        v[4 * j + 3] = f.w;
    }
    const unsigned long long anc = live ? a.anc[(int64_t)b * a.T + n] : 1ull;
    const int full = len / a.block_k;                                         // complete pages
    const int local = live ? (len + __popcll(anc) - 1) / a.block_k : 0;       // the node's own block
    const int past = min(full, local);                                        // candidates from the scan
    if (sub == 0 && lane < 4) s_draft[slot][lane] = 0u;
    if (sub == 0 && lane == 0) s_cnt[slot] = 0;
    __syncthreads();
    unsigned long long* list = s_list + (size_t)slot * WPR * kCap;
    if (live) {
        unsigned long long best = 0ull;
#pragma unroll
        for (int j = 0; j < kPerLane / 4; ++j) {
            const int c = 4 * (lane + 32 * sub) + 128 * WPR * j;
            if (__all_sync(0xffffffffu, c >= past)) break;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < past) best = max(best, cand_key(v[4 * j + e], c + e));
        }
        int rank = 0;
#pragma unroll
        for (int l = 0; l < 32; ++l) rank += __shfl_sync(0xffffffffu, best, l) > best;
        // lanes without candidates share the key 0 and the rank after the last candidate's
        const unsigned at = __ballot_sync(0xffffffffu, rank == K1 - 1 && best > 0);
        const unsigned long long bound = at ? __shfl_sync(0xffffffffu, best, __ffs(at) - 1) : 1ull;
#pragma unroll
        for (int j = 0; j < kPerLane / 4; ++j) {
            const int c = 4 * (lane + 32 * sub) + 128 * WPR * j;
            if (__all_sync(0xffffffffu, c >= past)) break;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < past) {
                    const unsigned long long k = cand_key(v[4 * j + e], c + e);
                    if (k >= bound) list[atomicAdd(&s_cnt[slot], 1)] = k;
                }
        }
        // blocks full .. local - 1: the cache's last tokens and the path's tokens that left them behind
        if (sub == 0 && local > full) {
            const int path = __popcll(anc);
            for (int m = lane; m < a.T; m += 32) {
                if (!((anc >> m) & 1)) continue;
                const int depth = __popcll(a.anc[(int64_t)b * a.T + m]) - 1;
                const int c = (len + depth) / a.block_k;
                if (c >= local || depth >= path) continue;
                const uint4* q = reinterpret_cast<const uint4*>(q_idx + (((int64_t)b * a.T + n) * a.H_kv + g) * a.d_idx);
                const uint4* k = reinterpret_cast<const uint4*>(k_idx + ((int64_t)b * a.T + m) * a.d_idx);
                float dot = 0.f;
                for (int x = 0; x < a.d_idx / 8; ++x) {
                    const uint4 qv = q[x], kv = k[x];
                    const __nv_bfloat162* qh = reinterpret_cast<const __nv_bfloat162*>(&qv);
                    const __nv_bfloat162* kh = reinterpret_cast<const __nv_bfloat162*>(&kv);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 qf = __bfloat1622float2(qh[e]), kf = __bfloat1622float2(kh[e]);
                        dot = fmaf(qf.x, kf.x, dot);
                        dot = fmaf(qf.y, kf.y, dot);
                    }
                }
                atomicMax(&s_draft[slot][c - full], (uint32_t)(cand_key(fmaxf(dot, -INFINITY), 0) >> 32));  // NaN: -inf
            }
            __syncwarp();
            for (int c = full + lane; c < local; c += 32) {
                uint32_t o = s_draft[slot][c - full];
                if (c == full && len % a.block_k) o = max(o, (uint32_t)(cand_key(vals[c], 0) >> 32));
                list[atomicAdd(&s_cnt[slot], 1)] = ((unsigned long long)o << 32) | (0xffffffffu - (uint32_t)c);
            }
        }
    }
    __syncthreads();
    const int take = min(a.topk, local);
    if (live) {
        const int cnt = s_cnt[slot];
        for (int i = sub * 32 + lane; i < cnt; i += WPR * 32) {
            const unsigned long long k = list[i];
            int rank = 0;
            for (int j = 0; j < cnt; ++j) rank += list[j] > k;
            if (rank < take) s_chosen[slot][rank] = (int)(0xffffffffu - (uint32_t)k);
            if (rank == a.topk - 1 || rank == a.topk) s_kth[slot][rank - a.topk + 1] = key_value(k);
        }
    }
    __syncthreads();
    if (!live_row || sub != 0) return;
    int32_t* out = a.blocks_out + gr * K1;
    if (!live) {
        if (lane < K1) out[lane] = -1;
        if (lane == 0 && a.margin_out) a.margin_out[gr] = INFINITY;
        return;
    }
    if (lane == 0 && a.margin_out)
        a.margin_out[gr] = local > a.topk ? (s_kth[slot][0] - s_kth[slot][1]) * a.scale_idx : INFINITY;
    // the chosen ids and the local block, ascending: each lane places its id by its rank
    const int mine = lane < take ? s_chosen[slot][lane] : (lane == take ? local : 0x7fffffff);
    int rank = 0;
    for (int x = 0; x <= take; ++x) rank += __shfl_sync(0xffffffffu, mine, x) < mine;
    if (lane <= take) out[rank] = mine;
    else if (lane < K1) out[lane] = -1;
}

}  // namespace

size_t tree_index_ws_bytes(int B, int N, int H_kv, int block_k, int T) {
    const size_t ld = ((size_t)(N + kScanTile - 1) / kScanTile) * (kScanTile / block_k);
    auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    return al((size_t)B * T * 8) + al((size_t)B * T * H_kv * ((ld + 3) / 4 * 4) * 4);
}
void tree_index_carve(TreeArgs* a, void* base) {
    const int ld = ((a->N + kScanTile - 1) / kScanTile) * (kScanTile / a->block_k);
    a->bmax_ld = (ld + 3) / 4 * 4;
    a->anc = static_cast<unsigned long long*>(base);
    a->bmax = reinterpret_cast<float*>(static_cast<uint8_t*>(base) + (((size_t)a->B * a->T * 8 + 255) & ~size_t(255)));
}

cudaError_t run_tree_index(const TreeArgs& a, const void* q_idx, const void* k_idx, const void* k_idx_pool, int num_sms,
                           cudaStream_t st) {
    const int R = a.T * a.H_kv;
    {
        CUtensorMap tq, tk;
        const int sw = a.d_idx * 2;
        if (!make_tmap_3d(&tq, q_idx, a.d_idx, R, a.B, (uint64_t)a.d_idx * 2, (uint64_t)R * a.d_idx * 2, a.d_idx, kTile, 1, sw) ||
            !make_tmap_2d(&tk, k_idx_pool, a.d_idx, (uint64_t)a.num_pages * a.block_k, (uint64_t)a.d_idx * 2, a.d_idx,
                          a.block_k, sw))
            return cudaErrorInvalidValue;
        ProfScope ps("tree_scan", st);
        auto launch = [&](auto kern, size_t bytes) -> cudaError_t {
            const size_t smem = bytes + 1024;
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            kern<<<dim3(num_sms, (R + 2 * kTile - 1) / (2 * kTile)), kScanThreads, smem, st>>>(tq, tk, a);
            return cudaGetLastError();
        };
        cudaError_t e;
        if (a.d_idx == 64)
            e = a.block_k == 128 ? launch(k_tree_scan<64, 128>, sizeof(TreeScanSmem<64>))
                : a.block_k == 64 ? launch(k_tree_scan<64, 64>, sizeof(TreeScanSmem<64>))
                                  : launch(k_tree_scan<64, 32>, sizeof(TreeScanSmem<64>));
        else
            e = a.block_k == 128 ? launch(k_tree_scan<32, 128>, sizeof(TreeScanSmem<32>))
                : a.block_k == 64 ? launch(k_tree_scan<32, 64>, sizeof(TreeScanSmem<32>))
                                  : launch(k_tree_scan<32, 32>, sizeof(TreeScanSmem<32>));
        if (e != cudaSuccess) return e;
    }
    ProfScope ps("tree_topk", st);
    const int64_t rows = (int64_t)a.B * R;
    const auto* q = static_cast<const __nv_bfloat16*>(q_idx);
    const auto* k = static_cast<const __nv_bfloat16*>(k_idx);
    // one warp per row while 16 candidates a lane suffice (512 blocks), or 64 (2048) when the rows fill the device;
    // else four warps, with as few candidates a lane as suffice (1024 rows of 2056 blocks: 14.8 us with room for 32, at
    // 64 the list's shared memory and 94 registers leave 5 CTAs an SM: 16.9 us)
    auto launch = [&](auto kern, int rpc) {
        return launch_pdl(kern, dim3((unsigned)((rows + rpc - 1) / rpc)), dim3(kTopkWarps * 32), 0, st, a, q, k);
    };
    if (a.bmax_ld <= 512) return launch(k_tree_topk<1, 16>, 4);
    if (a.bmax_ld <= 2048) return rows >= 16LL * num_sms ? launch(k_tree_topk<1, 64>, 4) : launch(k_tree_topk<4, 16>, 1);
    if (a.bmax_ld <= 4096) return launch(k_tree_topk<4, 32>, 1);
    return launch(k_tree_topk<4, 64>, 1);
}

}  // namespace msa
