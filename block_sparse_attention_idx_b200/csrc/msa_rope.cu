// Rotary positions (forward and gradient). A head's leading `rot` dims are rotated in pairs by the angle
// position * inv_freq[i] and scaled by amp; the rest is copied:
//   y_a = amp (x_a cos - x_b sin),  y_b = amp (x_a sin + x_b cos),  (a, b) = (i, i + rot/2) or (2i, 2i+1).
// The gradient applies the transposed map: the same with -sin.
//
// Angles. position * inv_freq reaches 1e6 radians and more, where 32 bits leave 0.06 radians of error, and 2^31, where a
// product in 64 bits leaves 2e-7. The angle is formed in turns, t = position * (inv_freq / 2 pi), both products as a sum of
// two 64-bit numbers (the rounding of a product is a fused multiply-add away), the whole turns are dropped and sincospif
// takes 2 (t - rint t) in about [-1, 1]: some ten 64-bit operations and one sincospif a pair, once per token and distinct
// table of frequencies (Q and K share one, Q_idx and K_idx another).
//
// HBM-bound: every element is read and written once. A CTA takes one token's heads of all tensors as a flat list of
// tasks (2V elements of a head, V pairs of one or two 16-byte loads each); a thread issues its loads, works out its share of
// the tables while they fly, then rotates. Resident warps are what covers the loads' latency: 16-bit inputs run best in small
// CTAs of 40 registers (32768 tokens of 64 + 4 heads of 128 and 4 + 1 of 64 dims, replayed: 196 us, 0.92 of the copy rate;
// before the angles were 128 bits wide 193 us, and then 198 us with 128 threads instead of 96, 253 us with 32 registers,
// 318 us with 90 and three tasks in flight, 299 us with a warp per token and tensor), 32-bit ones, twice the bytes a task, with
// up to 64 registers (8191 tokens: 102 us; 153 us with 40).
//
// V is the widest of 8, 4, 2, 1 that divides every tensor's rot / 2, so that a task lies in one half of a head. Narrower tasks
// are more instructions and requests for the same bytes: the same 32768 tokens take 200 us at V = 8, 268 at 4 (rot 120), 417
// at 2 (rot 124) and 625 at 1 (rot 126, or 128 with an odd half in the index heads alone); 8191 tokens in 32 bits 97, 99, 117
// and 181 us. One CTA shape serves all widths: one of 256 threads with four narrow tasks in flight took 651, 704 and 656 us
// (141, 134 and 174).
#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {

namespace {

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

// Threads of a CTA and CTAs an SM should hold, by element size.
template <typename TX>
struct RopeCta {
    static constexpr int kThreads = sizeof(TX) == 2 ? 96 : 192;
    static constexpr int kPerSm = sizeof(TX) == 2 ? 16 : 5;
};

// 2 t, t = pos * f / (2 pi) less its whole turns. Up to |pos * f| < 2^48 the low parts stay below 1/32 of a turn, and the
// result is that of the exact angle rounded to fp32.
__device__ __forceinline__ float rope_half_turns(double pos, double f) {
    constexpr double kTurn = 0.15915494309189535, kTurnLow = -9.839338337591243e-18;  // 1 / (2 pi)
    const double w = f * kTurn, w_low = fma(f, kTurn, -w) + f * kTurnLow;
    const double t = pos * w, t_low = fma(pos, w, -t) + pos * w_low;
    return (float)(2.0 * ((t - rint(t)) + t_low));
}

// gridDim.y CTAs share a token's tasks where the tokens alone are too few.
template <int V, bool IL, typename TX, typename TY>
__global__ void __launch_bounds__(RopeCta<TX>::kThreads, RopeCta<TX>::kPerSm) k_rope(const __grid_constant__ RopeArgs a) {
    __shared__ __align__(16) float s_cos[kRopeSegs * kMaxPairs], s_sin[kRopeSegs * kMaxPairs];
    const int64_t tok = blockIdx.x;
    const int nt = blockDim.x, part = (a.task0[a.nseg] + gridDim.y - 1) / gridDim.y;
    const int first = blockIdx.y * part, tasks = min(a.task0[a.nseg], first + part);
    for (int t = first + threadIdx.x; t - (int)threadIdx.x < tasks; t += nt) {
        Vec<TX, V> x0, x1;
        int seg = -1, oa, ob;  // segment (-1: nothing to do), offsets of the two halves within the token
        bool rot = false;
        if (t < tasks) {
            int s = 0;
            while (t >= a.task0[s + 1]) ++s;
            const RopeSeg& g = a.seg[s];
            const int i = t - a.task0[s], c = i & ((1 << g.lg) - 1), head = (i >> g.lg) * g.dim;
            rot = c < g.rot / (2 * V);
            if (rot || g.x != g.y) {  // (what is copied in place stays)
                seg = s;
                oa = head + (rot && !IL ? c * V : c * 2 * V);
                ob = oa + (rot && !IL ? g.rot / 2 : V);
                const TX* x = static_cast<const TX*>(g.x) + tok * g.x_stride;
                x0 = *reinterpret_cast<const Vec<TX, V>*>(x + oa);
                x1 = *reinterpret_cast<const Vec<TX, V>*>(x + ob);
            }
        }
        if (t == first + (int)threadIdx.x) {
            const double pos = a.positions ? (double)a.positions[tok] : (double)tok;
            for (int i = threadIdx.x; i < a.tab0[a.ntab]; i += nt) {
                int tab = 0;
                while (i >= a.tab0[tab + 1]) ++tab;
                const RopeSeg& g = a.seg[a.tab_seg[tab]];
                float sn, cn;
                sincospif(rope_half_turns(pos, g.inv_freq[i - a.tab0[tab]]), &sn, &cn);
                s_cos[tab * kMaxPairs + i - a.tab0[tab]] = cn * g.amp;
                s_sin[tab * kMaxPairs + i - a.tab0[tab]] = sn * (a.back ? -g.amp : g.amp);
            }
            __syncthreads();
        }
        if (seg < 0) continue;
        const RopeSeg& g = a.seg[seg];
        Vec<TY, V> y0, y1;
        // interleaved: pair e is elements 2e, 2e+1 of the 2V loaded ones (x0, then x1)
        auto in = [&](int i) { return to_f(i < V ? x0.v[i % V] : x1.v[i % V]); };
        auto out = [&](int i, float f) { (i < V ? y0.v[i % V] : y1.v[i % V]) = from_f<TY>(f); };
        if (rot) {
            const int at = g.tab * kMaxPairs + ((t - a.task0[seg]) & ((1 << g.lg) - 1)) * V;
            Vec<float, V> cn = *reinterpret_cast<const Vec<float, V>*>(s_cos + at);
            Vec<float, V> sn = *reinterpret_cast<const Vec<float, V>*>(s_sin + at);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int i0 = IL ? 2 * e : e, i1 = IL ? 2 * e + 1 : V + e;
                const float xa = in(i0), xb = in(i1);
                out(i0, xa * cn.v[e] - xb * sn.v[e]);
                out(i1, xa * sn.v[e] + xb * cn.v[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) out(e, in(e));
        }
        TY* y = static_cast<TY*>(g.y) + tok * g.y_stride;
        *reinterpret_cast<Vec<TY, V>*>(y + oa) = y0;
        *reinterpret_cast<Vec<TY, V>*>(y + ob) = y1;
    }
}

template <int V, bool IL>
cudaError_t launch_rope(const RopeArgs& a, bool x32, bool y32, cudaStream_t st) {
    const int nt = x32 ? RopeCta<float>::kThreads : RopeCta<__nv_bfloat16>::kThreads;
    const int64_t few = 4 * 148;  // CTAs: below, one pass of a CTA per part of a token
    const int passes = (a.task0[a.nseg] + nt - 1) / nt;
    const dim3 grid((unsigned)a.tokens, a.tokens >= few ? 1 : std::min<int64_t>(passes, (few + a.tokens - 1) / a.tokens));
    if (x32)
        y32 ? k_rope<V, IL, float, float><<<grid, nt, 0, st>>>(a) : k_rope<V, IL, float, __nv_bfloat16><<<grid, nt, 0, st>>>(a);
    else
        y32 ? k_rope<V, IL, __nv_bfloat16, float><<<grid, nt, 0, st>>>(a)
            : k_rope<V, IL, __nv_bfloat16, __nv_bfloat16><<<grid, nt, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t run_rope(RopeArgs a, bool interleaved, bool x32, bool y32, cudaStream_t st) {
    if (a.tokens <= 0) return cudaSuccess;
    // pairs of a task: the largest of 8, 4, 2, 1 that divides every segment's rot / 2 (odd sizes take narrower accesses)
    int v = 8;
    for (int s = 0; s < a.nseg; ++s)
        while (a.seg[s].rot / 2 % v != 0) v /= 2;
    a.ntab = a.task0[0] = a.tab0[0] = 0;
    for (int s = 0; s < a.nseg; ++s) {
        RopeSeg& g = a.seg[s];
        g.lg = 0;
        while ((2 * v << g.lg) < g.dim) ++g.lg;
        a.task0[s + 1] = a.task0[s] + (g.heads << g.lg);
        int t = 0;
        while (t < a.ntab && (a.seg[a.tab_seg[t]].inv_freq != g.inv_freq || a.seg[a.tab_seg[t]].rot != g.rot ||
                              a.seg[a.tab_seg[t]].amp != g.amp))
            ++t;
        g.tab = t;
        if (t == a.ntab) {
            a.tab_seg[t] = s;
            a.tab0[t + 1] = a.tab0[t] + g.rot / 2;
            ++a.ntab;
        }
    }
    ProfScope ps(a.back ? "rope_bwd" : "rope_fwd", st);
    switch (v) {
        case 8: return interleaved ? launch_rope<8, true>(a, x32, y32, st) : launch_rope<8, false>(a, x32, y32, st);
        case 4: return interleaved ? launch_rope<4, true>(a, x32, y32, st) : launch_rope<4, false>(a, x32, y32, st);
        case 2: return interleaved ? launch_rope<2, true>(a, x32, y32, st) : launch_rope<2, false>(a, x32, y32, st);
        default: return interleaved ? launch_rope<1, true>(a, x32, y32, st) : launch_rope<1, false>(a, x32, y32, st);
    }
}

}  // namespace msa
