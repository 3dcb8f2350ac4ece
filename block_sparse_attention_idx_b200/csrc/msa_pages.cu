// Paged K / V / K_idx caches: tokens written into their pages, and pages copied. A page holds one KV block
// (block_k tokens), so a selected block is one page: K, V [pages, block_k, H_kv, d], K_idx
// [pages, block_k, d_idx]. Token position p of sequence b lives in page page_table[b, p / block_k] at row
// p % block_k. Both kernels move bytes only and are HBM-bound (or, at decode sizes, one launch).
#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {

namespace {

// One warp per appended token: slot cache_len[b] + i gets row rows[b, i] (or i) of the new K, V and K_idx.
// A token is 2 H_kv d + d_idx elements (2.1 KB at H_kv = 4, d = 128): each lane issues all of its 16-byte
// loads of a tensor before the stores.
__global__ void __launch_bounds__(256) k_cache_append(const __grid_constant__ AppendArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int b = (int)(w / a.T_new), i = (int)(w - (int64_t)b * a.T_new);
    if (b >= a.B) return;
    const int n = a.n_new[b], len = a.cache_len[b];
    const bool bad_n = n < 0 || n > a.T_new || len < 0 || (n > 0 && len > a.N - n);
    if (bad_n && i == 0 && lane == 0 && a.status) raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xa01);
    if (i >= n || len < 0 || len > a.N - 1 - i) return;
    const int slot = len + i;
    const int page = a.page_table[(int64_t)b * a.cols + slot / a.block_k];
    const int row = a.rows ? a.rows[(int64_t)b * a.T_new + i] : i;
    if ((unsigned)page >= (unsigned)a.num_pages || (unsigned)row >= (unsigned)a.T) {
        if (lane == 0 && a.status) raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xa02);
        return;
    }
    const int64_t src = (int64_t)b * a.T + row, dst = (int64_t)page * a.block_k + slot % a.block_k;
    const uint4* k = a.k + src * a.kv_vec;
    const uint4* v = a.v + src * a.kv_vec;
    uint4* kp = a.k_pool + dst * a.kv_vec;
    uint4* vp = a.v_pool + dst * a.kv_vec;
    for (int x = lane; x < a.kv_vec; x += 64) {
        const bool two = x + 32 < a.kv_vec;
        const uint4 k0 = k[x], v0 = v[x];
        uint4 k1, v1;
        if (two) {
            k1 = k[x + 32];
            v1 = v[x + 32];
        }
        kp[x] = k0;
        vp[x] = v0;
        if (two) {
            kp[x + 32] = k1;
            vp[x + 32] = v1;
        }
    }
    if (lane < a.idx_vec) a.k_idx_pool[dst * a.idx_vec + lane] = a.k_idx[src * a.idx_vec + lane];
}

// One CTA per 16 KB piece of a copied page (K pieces, then V, then K_idx): 256 threads with four 16-byte
// loads in flight each.
constexpr int kPiece = 1024;  // 16-byte vectors

__global__ void __launch_bounds__(256) k_cache_copy_pages(const __grid_constant__ CopyArgs a) {
    const int per = 2 * a.kv_pieces + a.idx_pieces;
    const int i = blockIdx.x / per;
    int piece = blockIdx.x - i * per;
    const int src = a.src[i], dst = a.dst[i];
    if ((unsigned)src >= (unsigned)a.num_pages || (unsigned)dst >= (unsigned)a.num_pages) {
        if (piece == 0 && threadIdx.x == 0 && a.status) raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xa11);
        return;
    }
    if (src == dst) return;
    uint4* pool = a.k_pool;
    int64_t size = a.kv_vec;  // vectors of a page
    if (piece >= 2 * a.kv_pieces) {
        piece -= 2 * a.kv_pieces;
        pool = a.k_idx_pool;
        size = a.idx_vec;
    } else if (piece >= a.kv_pieces) {
        piece -= a.kv_pieces;
        pool = a.v_pool;
    }
    const uint4* from = pool + src * size + piece * kPiece;
    uint4* to = pool + dst * size + piece * kPiece;
    const int n = (int)min((int64_t)kPiece, size - (int64_t)piece * kPiece);
    uint4 r[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if ((int)threadIdx.x + 256 * x < n) r[x] = from[threadIdx.x + 256 * x];
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if ((int)threadIdx.x + 256 * x < n) to[threadIdx.x + 256 * x] = r[x];
}

}  // namespace

cudaError_t run_cache_append(const AppendArgs& a, cudaStream_t st) {
    const int64_t warps = (int64_t)a.B * a.T_new;
    if (warps <= 0) return cudaSuccess;
    ProfScope ps("cache_append", st);
    k_cache_append<<<(unsigned)((warps + 7) / 8), 256, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t run_cache_copy_pages(CopyArgs a, int n, cudaStream_t st) {
    if (n <= 0) return cudaSuccess;
    a.kv_pieces = (int)((a.kv_vec + kPiece - 1) / kPiece);
    a.idx_pieces = (int)((a.idx_vec + kPiece - 1) / kPiece);
    ProfScope ps("cache_copy_pages", st);
    k_cache_copy_pages<<<(unsigned)n * (2 * a.kv_pieces + a.idx_pieces), 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace msa
