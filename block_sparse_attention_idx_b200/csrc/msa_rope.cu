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
// c < rot / (2V), else 2V copied elements (skipped in place).
template <int V, bool IL, typename TX, typename TY>
__device__ __forceinline__ void rope_heads(const RopeSeg& g, int64_t tok, int h0, int h1, const float2* cs, int lane) {
    constexpr int U = V == 8 ? (sizeof(TX) == 2 ? 4 : 2) : 1;  // heads in flight
    const int cph = g.dim / (2 * V);                           // chunks per head, a power of two
    const int rc = g.rot / (2 * V);
    const TX* x = static_cast<const TX*>(g.x) + tok * g.x_stride;
    TY* y = static_cast<TY*>(g.y) + tok * g.y_stride;
    const bool in_place = g.x == g.y;
    const int n = (h1 - h0) * cph;
    for (int i0 = lane; i0 < n; i0 += 32 * U) {
        Vec<TX, V> a[U], b[U];
        int64_t oa[U], ob[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u;
            if (i >= n) break;
            const int c = i & (cph - 1);
            const int64_t head = (int64_t)(h0 + i / cph) * g.dim;
            const bool turn = c < rc;
            oa[u] = head + (turn && !IL ? c * V : c * 2 * V);
            ob[u] = oa[u] + (turn && !IL ? g.rot / 2 : V);
            a[u] = *reinterpret_cast<const Vec<TX, V>*>(x + oa[u]);
            b[u] = *reinterpret_cast<const Vec<TX, V>*>(x + ob[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u;
            if (i >= n) break;
            const int c = i & (cph - 1);
            Vec<TY, V> p, q;
            if (c < rc) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 t = cs[c * V + e];
                    // interleaved: pair e is elements 2e, 2e+1 of the 2V loaded ones (a, then b)
                    const float xa = to_f(IL ? (2 * e < V ? a[u].v[(2 * e) % V] : b[u].v[(2 * e) % V]) : a[u].v[e]);
                    const float xb = to_f(IL ? (2 * e + 1 < V ? a[u].v[(2 * e + 1) % V] : b[u].v[(2 * e + 1) % V])
                                             : b[u].v[e]);
                    const TY ya = from_f<TY>(xa * t.x - xb * t.y), yb = from_f<TY>(xa * t.y + xb * t.x);
                    if (IL) {
                        (2 * e < V ? p.v[(2 * e) % V] : q.v[(2 * e) % V]) = ya;
                        (2 * e + 1 < V ? p.v[(2 * e + 1) % V] : q.v[(2 * e + 1) % V]) = yb;
                    } else {
                        p.v[e] = ya;
                        q.v[e] = yb;
                    }
                }
            } else {
                if (in_place) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    p.v[e] = from_f<TY>(to_f(a[u].v[e]));
                    q.v[e] = from_f<TY>(to_f(b[u].v[e]));
                }
            }
            *reinterpret_cast<Vec<TY, V>*>(y + oa[u]) = p;
            *reinterpret_cast<Vec<TY, V>*>(y + ob[u]) = q;
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
