// Rotary positions (forward and gradient). A head's leading `rot` dims are rotated in pairs by the angle
// position * inv_freq[i] and scaled by amp; the rest is copied:
//   y_a = amp (x_a cos - x_b sin),  y_b = amp (x_a sin + x_b cos),  (a, b) = (i, i + rot/2) or (2i, 2i+1).
// The gradient applies the transposed map: the same with -sin.
//
// Angles. position * inv_freq reaches 1e6 radians, where 32 bits leave 0.06 radians of error. One lane per
// pair forms the angle in turns in 64 bits, t = position * (inv_freq / 2 pi), drops the whole turns and
// calls sincospif on 2 (t - rint t) in [-1, 1]: about four 64-bit operations and one sincospif a pair, once
// per (token, tensor), spread over a warp and shared by all heads through shared memory.
//
// HBM-bound: every element is read and written once. A warp takes one token of one tensor (or a slice of
// its heads when there are few tokens), so no block-wide barrier is needed; a lane owns V pairs, i.e. one
// or two 16-byte loads, of one column chunk and walks the heads with four (bf16) or two (fp32) heads'
// loads in flight.
#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {

namespace {

constexpr int kRopeWarps = 8;
constexpr int kMaxPairs = 64;  // dim <= 128

template <typename T, int N>
struct alignas(sizeof(T) * N >= 16 ? 16 : sizeof(T) * N) Vec {
    T v[N];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// The heads [h0, h1) of one token of one segment. Chunk c of a head holds 2V elements: V pairs for
// c < rot / (2V), else 2V copied elements (skipped in place). A lane keeps its chunk, and its V cosines and
// sines in registers, over all heads; 32 / chunks heads go side by side in a warp. (With the cosines read from
// shared memory for every head, 32768 tokens of 69 heads took 557 us.)
template <int V, bool IL, typename TX, typename TY>
__device__ __forceinline__ void rope_heads(const RopeSeg& g, int64_t tok, int h0, int h1, const float2* cs, int lane) {
    constexpr int U = V == 8 ? (sizeof(TX) == 2 ? 4 : 2) : 4;  // heads in flight
    const int dim = g.dim, rot = g.rot;
    const int lg = 31 - __clz(dim / (2 * V));  // log2 of the chunks per head
    const int cph = 1 << lg, lph = min(cph, 32), hstep = 32 / lph;
    const TX* x = static_cast<const TX*>(g.x) + tok * g.x_stride;
    TY* y = static_cast<TY*>(g.y) + tok * g.y_stride;
    for (int c = lane & (lph - 1); c < cph; c += 32) {
        const bool turn = c < rot / (2 * V);
        if (!turn && g.x == g.y) continue;
        float cn[V], sn[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 t = turn ? cs[c * V + e] : make_float2(1.f, 0.f);
            cn[e] = t.x;
            sn[e] = t.y;
        }
        const int oa = turn && !IL ? c * V : c * 2 * V, ob = oa + (turn && !IL ? rot / 2 : V);
        for (int h = h0 + lane / lph; h < h1; h += hstep * U) {
            Vec<TX, V> a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u * hstep < h1) {
                    a[u] = *reinterpret_cast<const Vec<TX, V>*>(x + (h + u * hstep) * dim + oa);
                    b[u] = *reinterpret_cast<const Vec<TX, V>*>(x + (h + u * hstep) * dim + ob);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u * hstep < h1) {
                    Vec<TY, V> p, q;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        // interleaved: pair e is elements 2e, 2e+1 of the 2V loaded ones (a, then b)
                        constexpr int W = V;
                        const int i0 = IL ? 2 * e : e, i1 = IL ? 2 * e + 1 : W + e;
                        const float xa = to_f(i0 < W ? a[u].v[i0 % W] : b[u].v[i0 % W]);
                        const float xb = to_f(i1 < W ? a[u].v[i1 % W] : b[u].v[i1 % W]);
                        // copied elements too: cos 1, sin 0, but without 0 * infinity
                        const float ya = turn ? xa * cn[e] - xb * sn[e] : xa, yb = turn ? xa * sn[e] + xb * cn[e] : xb;
                        (i0 < W ? p.v[i0 % W] : q.v[i0 % W]) = from_f<TY>(ya);
                        (i1 < W ? p.v[i1 % W] : q.v[i1 % W]) = from_f<TY>(yb);
                    }
                    *reinterpret_cast<Vec<TY, V>*>(y + (h + u * hstep) * dim + oa) = p;
                    *reinterpret_cast<Vec<TY, V>*>(y + (h + u * hstep) * dim + ob) = q;
                }
        }
    }
}

template <bool IL, typename TX, typename TY>
__global__ void __launch_bounds__(kRopeWarps * 32) k_rope(const __grid_constant__ RopeArgs a) {
    __shared__ float2 s_cs[kRopeWarps][kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t wid = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t tok = wid / a.units;
    if (tok >= a.tokens) return;
    const int unit = (int)(wid - tok * a.units);
    int s = 0;
    while (s + 1 < a.nseg && unit >= a.unit0[s + 1]) ++s;
    const RopeSeg& g = a.seg[s];
    const int h0 = (unit - a.unit0[s]) * g.heads_per_unit, h1 = min(g.heads, h0 + g.heads_per_unit);
    const double pos = a.positions ? (double)a.positions[tok] : (double)tok;
    for (int i = lane; i < g.rot / 2; i += 32) {
        const double t = pos * (g.inv_freq[i] * 0.15915494309189535);  // turns: 1 / (2 pi)
        float sn, cn;
        sincospif((float)(2.0 * (t - rint(t))), &sn, &cn);
        s_cs[warp][i] = make_float2(cn * g.amp, sn * (a.back ? -g.amp : g.amp));
    }
    __syncwarp();
    switch (g.vec) {
        case 8: rope_heads<8, IL, TX, TY>(g, tok, h0, h1, s_cs[warp], lane); break;
        case 4: rope_heads<4, IL, TX, TY>(g, tok, h0, h1, s_cs[warp], lane); break;
        case 2: rope_heads<2, IL, TX, TY>(g, tok, h0, h1, s_cs[warp], lane); break;
        default: rope_heads<1, IL, TX, TY>(g, tok, h0, h1, s_cs[warp], lane);
    }
}

template <bool IL>
cudaError_t launch_rope(const RopeArgs& a, bool x32, bool y32, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.tokens * a.units + kRopeWarps - 1) / kRopeWarps);
    if (x32)
        y32 ? k_rope<IL, float, float><<<grid, kRopeWarps * 32, 0, st>>>(a)
            : k_rope<IL, float, __nv_bfloat16><<<grid, kRopeWarps * 32, 0, st>>>(a);
    else
        y32 ? k_rope<IL, __nv_bfloat16, float><<<grid, kRopeWarps * 32, 0, st>>>(a)
            : k_rope<IL, __nv_bfloat16, __nv_bfloat16><<<grid, kRopeWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t run_rope(RopeArgs a, bool interleaved, bool x32, bool y32, int num_sms, cudaStream_t st) {
    if (a.tokens <= 0) return cudaSuccess;
    // heads of a unit: 32 (or 64-dim: 64) heads in 8 passes of a warp, halved while the launch has fewer
    // than 8 warps an SM, so that few tokens still spread over the device
    int slice = 256;  // chunks of 16 elements per unit
    for (;; slice /= 2) {
        a.units = 0;
        for (int s = 0; s < a.nseg; ++s) {
            RopeSeg& g = a.seg[s];
            g.heads_per_unit = std::max(1, slice * 16 / g.dim);
            a.unit0[s] = a.units;
            a.units += (g.heads + g.heads_per_unit - 1) / g.heads_per_unit;
        }
        if (slice <= 32 || a.tokens * a.units >= 8LL * num_sms) break;
    }
    if ((a.tokens * a.units + kRopeWarps - 1) / kRopeWarps > 0x7fffffffLL) return cudaErrorInvalidValue;
    ProfScope ps(a.back ? "rope_bwd" : "rope_fwd", st);
    return interleaved ? launch_rope<true>(a, x32, y32, st) : launch_rope<false>(a, x32, y32, st);
}

}  // namespace msa
