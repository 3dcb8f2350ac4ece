// Paged K / V / K_idx caches: tokens written into their pages, and pages copied. A page holds one KV block
// (block_k tokens), so a selected block is one page: K, V [pages, block_k, H_kv, d], K_idx
// [pages, block_k, d_idx]. Token position p of sequence b lives in page page_table[b, p / block_k] at row
// p % block_k. Both kernels move bytes only and are HBM-bound (or, at decode sizes, one launch).
#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {

namespace {

// One warp per appended token: slot cache_len[b] + i gets row rows[b, i] (or i) of the new K, V and K_idx. A token is
// 2 H_kv d + d_idx elements (2.1 KB at H_kv = 4, d = 128). Its loads are issued before its slot is known: they need the
// row only, and the chain length -> page -> store is as long as they are. The price: a warp past its sequence's n_new has read a
// row that it drops. 16 x 1024 rows of which three quarters are new: 35.7 MB read where 27 MB are written, 14.2 us, 0.58 of
// the copy rate (4 CTAs an SM at 58 registers, 3.5 waves of them); at 64 x 16 rows it is one short launch either way.
__global__ void __launch_bounds__(256) k_cache_append(const __grid_constant__ AppendArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int b = (int)(w / a.T_new), i = (int)(w - (int64_t)b * a.T_new);
    if (b >= a.B) return;
    const int row = a.rows ? a.rows[(int64_t)b * a.T_new + i] : i;
    const int n = a.n_new[b], len = a.cache_len[b];
    const bool row_ok = (unsigned)row < (unsigned)a.T;
    const int64_t src = (int64_t)b * a.T + (row_ok ? row : 0);
    uint4 k[4], v[4], ki;  // H_kv d <= 1024 elements: up to 4 vectors a lane
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if (lane + 32 * x < a.kv_vec) {
            k[x] = a.k[src * a.kv_vec + lane + 32 * x];
            v[x] = a.v[src * a.kv_vec + lane + 32 * x];
        }
    if (lane < a.idx_vec) ki = a.k_idx[src * a.idx_vec + lane];
    const bool bad_n = n < 0 || n > a.T_new || len < 0 || (n > 0 && len > a.N - n);
    if (bad_n && i == 0 && lane == 0 && a.status) raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xa01);
    if (i >= n || len < 0 || len > a.N - 1 - i) return;
    const int slot = len + i;
    const int page = a.page_table[(int64_t)b * a.cols + slot / a.block_k];
    if ((unsigned)page >= (unsigned)a.num_pages || !row_ok) {
        if (lane == 0 && a.status) raise_flag(a.status, MSA_DEV_BAD_BLOCK, 0xa02);
        return;
    }
    const int64_t dst = (int64_t)page * a.block_k + slot % a.block_k;
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if (lane + 32 * x < a.kv_vec) {
            a.k_pool[dst * a.kv_vec + lane + 32 * x] = k[x];
            a.v_pool[dst * a.kv_vec + lane + 32 * x] = v[x];
        }
    if (lane < a.idx_vec) a.k_idx_pool[dst * a.idx_vec + lane] = ki;
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
