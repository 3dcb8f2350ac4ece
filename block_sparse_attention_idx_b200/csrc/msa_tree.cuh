// What the selection and the attention of drafted-token trees share: lengths as the kernels read them, the
// page lookup and the ancestor sets.
#pragma once
#include <algorithm>

#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {

namespace {

// Launch after the previous kernel of the stream with programmatic serialisation (see pdl_wait).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

constexpr int kTile = 128;  // keys of a tile: 128 / block_k pages

// Lengths as every kernel reads them: clamped into range, so that no value indexes past a buffer (the
// Top-k and attention kernels report a value outside).
__device__ __forceinline__ int tree_len(const TreeArgs& a, int b) { return min(max(a.cache_len[b], 0), a.N); }
__device__ __forceinline__ int tree_nodes(const TreeArgs& a, int b) { return min(max(a.n_nodes[b], 0), a.T); }
__device__ __forceinline__ int scan_tiles(const TreeArgs& a, int b) {
    return tree_nodes(a, b) > 0 ? (tree_len(a, b) + kTile - 1) / kTile : 0;
}
// Page of block c of sequence b; an id outside the pool reads page 0 and is reported.
__device__ __forceinline__ int tree_page(const TreeArgs& a, int b, int c, unsigned where) {
    const int p = a.page_table[(int64_t)b * a.cols + c];
    if ((unsigned)p < (unsigned)a.num_pages) return p;
    raise_flag(a.status, MSA_DEV_BAD_BLOCK, where);
    return 0;
}

// Ancestor sets (bit m of anc[n]: node m is n or an ancestor of n) of the `nodes` <= 64 nodes of sequence
// b by pointer doubling: six rounds of anc[n] |= anc[up[n]], up[n] = up[up[n]]. Called by threads 0..63 (two
// full warps), which meet at named barrier `bar`. A parent outside [-1, n) counts as -1 and is reported.
__device__ void tree_ancestors(const TreeArgs& a, int b, int nodes, unsigned long long* anc, int* up, uint32_t bar,
                               unsigned where) {
    const int n = threadIdx.x & 63;
    int p = -1;
    if (n < nodes) {
        p = a.parents[(int64_t)b * a.T + n];
        if (p < -1 || p >= n) {
            raise_flag(a.status, MSA_DEV_BAD_BLOCK, where);
            p = -1;
        }
    }
    unsigned long long m = 1ull << n;
    anc[n] = m;
    up[n] = p;
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        bar_sync_named(bar, 64);
        unsigned long long mm = 0ull;
        int pp = -1;
        if (p >= 0) {
            mm = anc[p];
            pp = up[p];
        }
        bar_sync_named(bar, 64);
        m |= mm;
        p = pp;
        anc[n] = m;
        up[n] = p;
    }
    bar_sync_named(bar, 64);
}

}  // namespace

}  // namespace msa
