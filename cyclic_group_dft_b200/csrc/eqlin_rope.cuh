// eqlin_rope.cuh -- rotary positions with several axes on equivariant features.
//
// A head is Dh channels of G group elements.  Channel c and channel c + Dh/2 form pair c; the
// pairs are divided among the axes in order, n_a of them for axis a, and pair j of axis a turns
// by angle = position[n, a] * base^(-j / n_a):
//     y[c]        = x[c] cos - x[c + Dh/2] sin
//     y[c + Dh/2] = x[c + Dh/2] cos + x[c] sin
// for every group element alike, so the rotation commutes with shifts of the group axis.  The
// inverse rotation (sin negated) is also the gradient.
//
// The angle is reduced exactly: a frequency is held in turns as a 64-bit binary fraction F
// (error below 2^-64 turns), position * F wraps modulo one turn in integer arithmetic, and its
// top 32 bits, rounded to the 24 of an fp32 number, give the angle within 2^-26 turns for every 32-bit position (half a
// unit of fp32 just below half a turn).  An fp32 product would
// lose 2^-24 of the whole angle, which is several percent of a turn at position 10^6.
//
// Bound by memory: one read and one write of the features.  A block takes a few tokens,
// computes their cos and sin once into shared memory for all heads, and rotates whole vectors.
// bf16, 200704 tokens, 6 heads of 32 channels, G = 4: 105 us for 618 MB (5.9 TB/s).
#pragma once

#include "eqlin_vec.cuh"
#include "sm100_ptx.cuh"

namespace eqlin {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;
constexpr int kMaxAxes = 4;
constexpr int kUnroll = 4;          // vector pairs in flight per thread
constexpr int kMaxSmemPairs = 4096; // tokens of a block * pairs

struct Params {
    const void* x;
    void* y;
    const int32_t* positions;      // [N, axes]
    long long N, x_stride, y_stride;
    int heads, pairs, half, lg_g;  // half = pairs * G features
    int axes, tokens;              // tokens per block
    int section_end[kMaxAxes];     // first pair past each axis
    float sign;                    // -1: inverse
    unsigned long long turns[kMaxPairs];
};

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads, 3) eqlin_rope_kernel(const __grid_constant__ Params p) {
    using V = Vec<T, VEC>;
    extern __shared__ float2 cs[];   // [tokens][pairs]: cos, sin
    const long long first = static_cast<long long>(blockIdx.x) * p.tokens;
    const int here = static_cast<int>(p.N - first < p.tokens ? p.N - first : p.tokens);
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int nv = p.half / VEC;               // vectors of half a head
    const int per_token = p.heads * nv, total = here * per_token;
    const T* x = static_cast<const T*>(p.x) + first * p.x_stride;
    T* y = static_cast<T*>(p.y) + first * p.y_stride;
    typename V::Raw lo[kUnroll], hi[kUnroll];
    int tok[kUnroll], feat[kUnroll];           // token of the block, feature of the row
    auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads;
            tok[u] = i / per_token;
            const int r = i - tok[u] * per_token, h = r / nv;
            feat[u] = r * VEC + h * p.half;    // h heads of 2 * half, of which r counts half
            if (i < total) {
                const T* at = x + tok[u] * p.x_stride + feat[u];
                lo[u] = V::load(at);
                hi[u] = V::load(at + p.half);
            }
        }
    };
    fetch(threadIdx.x);                        // on their way while the angles are computed
    for (int i = threadIdx.x; i < here * p.pairs; i += kThreads) {
        const int t = i / p.pairs, j = i - t * p.pairs;
        int a = 0;
        while (a + 1 < p.axes && j >= p.section_end[a]) ++a;
        const long long pos = p.positions[(first + t) * p.axes + a];
        const unsigned long long phase = static_cast<unsigned long long>(pos) * p.turns[j];
        const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * (1.f / 2147483648.f);
        float s, c;
        sincospif(half_turns, &s, &c);
        cs[i] = make_float2(c, s * p.sign);
    }
    __syncthreads();
    for (int i0 = threadIdx.x; i0 < total;) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (i0 + u * kThreads >= total) break;
            float a[VEC], b[VEC], ya[VEC], yb[VEC];
            V::unpack(lo[u], a);
            V::unpack(hi[u], b);
            const float2* t = cs + tok[u] * p.pairs;
            const int in_half = feat[u] % p.half;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 w = t[(in_half + e) >> p.lg_g];
                ya[e] = a[e] * w.x - b[e] * w.y;
                yb[e] = b[e] * w.x + a[e] * w.y;
            }
            T* to = y + tok[u] * p.y_stride + feat[u];
            V::store(to, V::pack(ya));
            V::store(to + p.half, V::pack(yb));
        }
        i0 += kThreads * kUnroll;
        if (i0 < total) fetch(i0);
    }
}

}  // namespace rope
}  // namespace eqlin
