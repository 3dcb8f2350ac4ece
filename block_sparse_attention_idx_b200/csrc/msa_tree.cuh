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

// One lane of a converged warp; the loops that issue TMA copies and MMAs run warp-uniform around it.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

constexpr int kTile = 128;  // rows of a product, and keys of an attention tile (128 / block_k pages)

// Lengths as every kernel reads them: clamped into range, so that no value indexes past a buffer (the
// Top-k and attention kernels report a value outside).
__device__ __forceinline__ int tree_len(const TreeArgs& a, int b) { return min(max(a.cache_len[b], 0), a.N); }
__device__ __forceinline__ int tree_nodes(const TreeArgs& a, int b) { return min(max(a.n_nodes[b], 0), a.T); }
// Page of block c of sequence b; an id outside the pool reads page 0 and is reported.
__device__ __forceinline__ int tree_page(const TreeArgs& a, int b, int c, unsigned where) {
    const int p = a.page_table[(int64_t)b * a.cols + c];
    if ((unsigned)p < (unsigned)a.num_pages) return p;
    raise_flag(a.status, MSA_DEV_BAD_BLOCK, where);
    return 0;
}

// Ancestor sets of the `nodes` <= 64 nodes of sequence b, by the 32 lanes of one warp: lane l gets the sets
// of nodes l and l + 32 (bit m: node m is the node itself or an ancestor; a node that does not exist has only
// its own bit). Pointer doubling in registers: anc[n] |= anc[up[n]], up[n] = up[up[n]], as often as paths of
// T nodes need. A parent outside [-1, n) counts as -1 and is reported. p0, p1: the parents as loaded.
__device__ __forceinline__ void tree_ancestors(const TreeArgs& a, int nodes, int p0, int p1, unsigned long long (&anc)[2],
                                               unsigned where) {
    const int lane = threadIdx.x & 31;
    int up[2] = {lane < nodes ? p0 : -1, lane + 32 < nodes ? p1 : -1};
    bool bad = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if (up[x] < -1 || up[x] >= lane + 32 * x) {
            bad = true;
            up[x] = -1;
        }
        anc[x] = 1ull << (lane + 32 * x);
    }
    if (bad) raise_flag(a.status, MSA_DEV_BAD_BLOCK, where);
    for (int span = 1; span < a.T; span *= 2) {
        unsigned long long na[2];
        int nu[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int u = up[x];
            const unsigned long long lo = __shfl_sync(0xffffffffu, anc[0], u & 31), hi = __shfl_sync(0xffffffffu, anc[1], u & 31);
            const int ul = __shfl_sync(0xffffffffu, up[0], u & 31), uh = __shfl_sync(0xffffffffu, up[1], u & 31);
            na[x] = u < 0 ? 0ull : u < 32 ? lo : hi;
            nu[x] = u < 0 ? -1 : u < 32 ? ul : uh;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            anc[x] |= na[x];
            up[x] = nu[x];
        }
    }
}
__device__ __forceinline__ int load_parent(const TreeArgs& a, int b, int n) {
    return n < a.T ? a.parents[(int64_t)b * a.T + n] : -1;
}

}  // namespace

}  // namespace msa
