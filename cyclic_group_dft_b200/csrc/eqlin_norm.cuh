// eqlin_norm.cuh -- root-mean-square norm of equivariant features with the residual's
// addition, its 8-bit output and its gradients.
//
// For a token row r = x + residual of L = C * G features (group axis fastest):
//     rstd = 1 / sqrt(mean(r^2) + eps),   y[c,g] = r[c,g] * rstd * w[c]
// The mean runs over channels and group elements and w is shared over the group axis, so a
// cyclic shift of the group axis shifts y.  With u = r * rstd and upstream gradients dy (of y)
// and dsum (of r through the residual stream):
//     dr = dsum + rstd * (w dy - u * mean(w dy u)),   dw[c] = sum_{n,g} dy u
//
// Bound by memory: each tensor crosses HBM once.  A row is held in registers by a group of
// threads (VPT vectors each), so the statistics and the output come from one read.  The
// weights of a thread's columns are loaded once and kept for all rows that the thread's
// group visits; dw is summed in registers over those rows, then over the block's groups and
// the group axis, written per block, and reduced over blocks in a fixed order in float64.
//
// bf16, 200704 tokens of 96 channels, G = 4 (154 MB a tensor): forward 110 us for four tensors (5.6 TB/s), gradients
// 82 us for three (5.6 TB/s), with dsum 110 us for four.  8-bit output, 25088 tokens of 64 channels, G = 8: 18.7 us (4.8
// TB/s).  Wide rows, 12544 of 4096 features: forward 68 us for 411 MB (6.1 TB/s), gradients 85.
#pragma once

#include <cfloat>

#include <cuda_fp8.h>

#include "eqlin_vec.cuh"
#include "sm100_ptx.cuh"

namespace eqlin {
namespace norm {

constexpr int kThreads = 256;      // block of the narrow form: 256 / TPR row groups
constexpr int kMaxWide = 512;      // the wide form: one row group of 64..512 threads
constexpr int kMaxVpt = 4;
constexpr float kE4m3Max = 448.f;
// Blocks on an SM, by the vectors of a thread: what the registers allow (the gradients hold three tensors' vectors
// and the sums of dw).  Grids are this many blocks for each SM, so that all run at once.
constexpr int fwd_blocks(int vpt, bool wide) { return wide ? (vpt <= 2 ? 2 : 1) : vpt == 1 ? 6 : vpt == 2 ? 4 : 3; }
constexpr int bwd_blocks(int vpt, bool wide) { return wide ? (vpt <= 2 ? 2 : 1) : vpt == 1 ? 4 : vpt == 2 ? 3 : 2; }

__device__ __forceinline__ void cp_async16(uint4* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}

struct Params {
    const void* x;          // fwd: x;  bwd: dy
    const void* residual;   // fwd: residual or NULL;  bwd: the stored sum r
    const void* weight;     // [C] or NULL (ones)
    void* y;                // fwd: y;  bwd: dx
    void* sum;              // fwd: r or NULL;  bwd: dsum or NULL (read)
    float* scale;           // 8-bit form: row scales
    float* partial;         // bwd: [blocks][C] sums of dw, or NULL
    long long N;
    int L, C, lg_g;         // features of a row, channels, log2(G)
    int tpr;                // threads of a row group (a power of two)
    int w_dtype;
    float eps;
};

// Sum of `v` over the tpr threads of a row group, the same bits in each of them: butterfly
// shuffles within a warp, then (wide form) the warps' sums added in warp order.
template <bool WIDE, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], int tpr, float* red) {
    const int lanes = WIDE ? 32 : tpr;
    for (int o = lanes >> 1; o > 0; o >>= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    }
    if constexpr (WIDE) {
        const int warps = tpr >> 5;
        __syncthreads();   // the previous use of red is over
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) red[k * 16 + (threadIdx.x >> 5)] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = 0.f;
            for (int w = 0; w < warps; ++w) v[k] += red[k * 16 + w];
        }
    }
}
template <bool WIDE>
__device__ __forceinline__ float group_max(float v, int tpr, float* red) {
    const int lanes = WIDE ? 32 : tpr;
    for (int o = lanes >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if constexpr (WIDE) {
        const int warps = tpr >> 5;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        for (int w = 0; w < warps; ++w) v = fmaxf(v, red[w]);
    }
    return v;
}

template <int VEC, int VPT>
__device__ __forceinline__ void load_weights(const Params& p, int lane, float (&w)[VPT][VEC]) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int at = (lane + j * p.tpr) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            w[j][e] = (p.weight && at + e < p.L) ? load_param(p.weight, p.w_dtype, (at + e) >> p.lg_g) : 1.f;
    }
}

// The forward.  OUT8: y in e4m3 with one scale per row, scale = max|y| / 448 (1 for a row of
// zeros), y8 = e4m3(y / scale) rounded to nearest even.  x, residual, y and sum may be the
// same tensor: every thread reads its elements of a row before any of them is written.
// The dependent launch is let go at the start: its griddepcontrol.wait still waits for the
// end of this grid.
template <class T, int VEC, int VPT, bool WIDE, bool OUT8>
__global__ void __launch_bounds__(WIDE ? kMaxWide : kThreads, fwd_blocks(VPT, WIDE)) eqlin_add_rmsnorm_kernel(const Params p) {
    using V = Vec<T, VEC>;
    __shared__ float red[16];
    const int groups = WIDE ? 1 : kThreads / p.tpr;
    const int lane = WIDE ? threadIdx.x : threadIdx.x & (p.tpr - 1);
    const int group = WIDE ? 0 : threadIdx.x / p.tpr;
    const int nv = p.L / VEC;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    float w[VPT][VEC];
    load_weights<VEC, VPT>(p, lane, w);
    const float inv_l = 1.f / static_cast<float>(p.L);
    // the loop bound is uniform over the block, so the shuffles and barriers of the
    // reductions are reached by every thread; groups past the last row do no memory access
    for (long long base = static_cast<long long>(blockIdx.x) * groups; base < p.N;
         base += static_cast<long long>(gridDim.x) * groups) {
        const long long row = base + group;
        const bool live = row < p.N;
        const T* x = static_cast<const T*>(p.x) + row * p.L;
        const T* res = static_cast<const T*>(p.residual) + row * p.L;
        typename V::Raw rx[VPT], rr[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = lane + j * p.tpr;
            rx[j] = typename V::Raw{};
            rr[j] = typename V::Raw{};
            if (live && v < nv) {
                rx[j] = V::load(x + v * VEC);
                if (p.residual) rr[j] = V::load(res + v * VEC);
            }
        }
        float r[VPT][VEC];
        float ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float a[VEC], b[VEC];
            V::unpack(rx[j], a);
            V::unpack(rr[j], b);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                r[j][e] = p.residual ? a[e] + b[e] : a[e];
                ss[0] = fmaf(r[j][e], r[j][e], ss[0]);
            }
        }
        group_sum<WIDE, 1>(ss, p.tpr, red);
        const float rstd = 1.f / sqrtf(fmaf(ss[0], inv_l, p.eps));
        if (p.sum && live) {
            T* out = static_cast<T*>(p.sum) + row * p.L;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = lane + j * p.tpr;
                if (v < nv) V::store(out + v * VEC, V::pack(r[j]));
            }
        }
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                r[j][e] = r[j][e] * rstd * w[j][e];
                if constexpr (OUT8) top = fmaxf(top, fabsf(r[j][e]));
            }
        if constexpr (OUT8) {
            top = group_max<WIDE>(top, p.tpr, red);
            float scale = top > 0.f ? top / kE4m3Max : 1.f, up = 1.f;
            if (scale < FLT_MIN) {
                // Its reciprocal would be infinite: scale and row times 2^64 instead.  Rounded up, so that it is
                // not 0 and y / scale not above 448.
                scale = __fdiv_ru(top, kE4m3Max);
                up = 18446744073709551616.f;
#pragma unroll
                for (int j = 0; j < VPT; ++j)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) r[j][e] *= up;
            }
            if (!live) continue;
            // one reciprocal for the row: within 2 units in the last place of y / scale, far below half of an
            // e4m3 step (quotients instead: 25088 rows of 512 features 17 to 22 us, 200704 of 384 85 to 105)
            const float inv = 1.f / (scale * up);
            if (lane == 0) p.scale[row] = scale;
            uint8_t* out = static_cast<uint8_t*>(p.y) + row * p.L;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = lane + j * p.tpr;
                if (v >= nv) continue;
                if constexpr (VEC == 1) {
                    out[v] = __nv_cvt_float_to_fp8(r[j][0] * inv, __NV_SATFINITE, __NV_E4M3);
                } else {
                    uint32_t q[VEC / 4];
#pragma unroll
                    for (int e = 0; e < VEC; e += 4) {
                        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(r[j][e] * inv, r[j][e + 1] * inv),
                                                                    __NV_SATFINITE, __NV_E4M3);
                        const uint32_t b = __nv_cvt_float2_to_fp8x2(
                            make_float2(r[j][e + 2] * inv, r[j][e + 3] * inv), __NV_SATFINITE, __NV_E4M3);
                        q[e / 4] = a | (b << 16);
                    }
                    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(out + v * VEC) = make_uint2(q[0], q[1]);
                    else *reinterpret_cast<uint32_t*>(out + v * VEC) = q[0];
                }
            }
        } else if (live) {
            T* out = static_cast<T*>(p.y) + row * p.L;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = lane + j * p.tpr;
                if (v < nv) V::store(out + v * VEC, V::pack(r[j]));
            }
        }
    }
}

// The gradients: dx (of x and of the residual alike) and, per block, the sums of dw.
// Dynamic shared memory: the weights of tpr * VPT * VEC columns (registers would cost a block per SM); behind them
// first the ring of the next row's vectors, then groups * tpr * VPT * VEC floats for the sums of dw.
// RING (narrow form, vectors of 16 bytes, no dsum): a thread copies its vectors of the group's next row asynchronously
// while it works on this one, and reads back its own alone, so that no barrier is needed.  200704 tokens of 96
// channels, G = 4: 82 us for 98.  With dsum three tensors in flight are enough without it, and the ring was slower
// (forward and gradients 220 us for 210).
template <class T, int VEC, int VPT, bool WIDE, bool RING>
__global__ void __launch_bounds__(WIDE ? kMaxWide : kThreads, bwd_blocks(VPT, WIDE)) eqlin_rmsnorm_bwd_kernel(const Params p) {
    using V = Vec<T, VEC>;
    __shared__ float red[32];
    extern __shared__ __align__(16) float w_smem[];
    float* acc_smem = w_smem + p.tpr * VPT * VEC;
    const int groups = WIDE ? 1 : kThreads / p.tpr;
    const int lane = WIDE ? threadIdx.x : threadIdx.x & (p.tpr - 1);
    const int group = WIDE ? 0 : threadIdx.x / p.tpr;
    const int nv = p.L / VEC;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    float dw[VPT][VEC];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[j][e] = 0.f;
    for (int i = threadIdx.x; i < p.tpr * VPT * VEC; i += blockDim.x)
        w_smem[i] = p.weight && i < p.L ? load_param(p.weight, p.w_dtype, i >> p.lg_g) : 1.f;
    __syncthreads();
    auto weights = [&](int j, float (&w)[VEC]) {
        const float* s = w_smem + (lane + j * p.tpr) * VEC;
        if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int e = 0; e < VEC; e += 4) {
                const float4 v = *reinterpret_cast<const float4*>(s + e);
                w[e] = v.x;
                w[e + 1] = v.y;
                w[e + 2] = v.z;
                w[e + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = s[e];
        }
    };
    const float inv_l = 1.f / static_cast<float>(p.L);
    const long long step = static_cast<long long>(gridDim.x) * groups;
    uint4* ring = reinterpret_cast<uint4*>(acc_smem) + threadIdx.x;
    auto slot = [&](int stage, int tensor, int j) { return ring + ((stage * 2 + tensor) * VPT + j) * kThreads; };
    auto fetch = [&](long long row, int stage) {
        if constexpr (RING) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = lane + j * p.tpr;
                if (row >= p.N || v >= nv) continue;
                const long long at = row * p.L + v * VEC;
                cp_async16(slot(stage, 0, j), static_cast<const T*>(p.x) + at);
                cp_async16(slot(stage, 1, j), static_cast<const T*>(p.residual) + at);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    int stage = 0;
    fetch(static_cast<long long>(blockIdx.x) * groups + group, 0);
    for (long long base = static_cast<long long>(blockIdx.x) * groups; base < p.N; base += step, stage ^= 1) {
        const long long row = base + group;
        const bool live = row < p.N;
        typename V::Raw rdy[VPT], rs[VPT], rd[VPT];
        if constexpr (RING) {
            fetch(row + step, stage ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = lane + j * p.tpr;
            rdy[j] = rs[j] = rd[j] = typename V::Raw{};
            if (live && v < nv) {
                if constexpr (RING) {
                    rdy[j] = *slot(stage, 0, j);
                    rs[j] = *slot(stage, 1, j);
                } else {
                    const long long at = row * p.L + v * VEC;
                    rdy[j] = V::load(static_cast<const T*>(p.x) + at);
                    rs[j] = V::load(static_cast<const T*>(p.residual) + at);
                    if (p.sum) rd[j] = V::load(static_cast<const T*>(p.sum) + at);
                }
            }
        }
        float s[2] = {0.f, 0.f};   // sum r^2 and sum w dy r
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float dy[VEC], r[VEC], w[VEC];
            V::unpack(rdy[j], dy);
            V::unpack(rs[j], r);
            weights(j, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s[0] = fmaf(r[e], r[e], s[0]);
                s[1] = fmaf(w[e] * dy[e], r[e], s[1]);
            }
        }
        group_sum<WIDE, 2>(s, p.tpr, red);
        // places past the last row hold zeros and must add none to dw: with eps = 0 they would have an infinite rstd
        const float rstd = live ? 1.f / sqrtf(fmaf(s[0], inv_l, p.eps)) : 0.f;
        const float inner = s[1] * inv_l * rstd * rstd;   // mean(w dy u) * rstd, for u = r * rstd
        T* out = static_cast<T*>(p.y) + row * p.L;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = lane + j * p.tpr;
            float dy[VEC], r[VEC], d[VEC], w[VEC];
            V::unpack(rdy[j], dy);
            V::unpack(rs[j], r);
            V::unpack(rd[j], d);
            weights(j, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                dw[j][e] = fmaf(dy[e], r[e] * rstd, dw[j][e]);
                d[e] += rstd * (w[e] * dy[e] - r[e] * inner);
            }
            if (live && v < nv) V::store(out + v * VEC, V::pack(d));
        }
    }
    if (!p.partial) return;
    if constexpr (RING) asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();   // the ring is read
    const int row_pad = p.tpr * VPT * VEC;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            acc_smem[group * row_pad + (lane + j * p.tpr) * VEC + e] = dw[j][e];
    __syncthreads();
    const int G = 1 << p.lg_g;
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
        float sum = 0.f;
        for (int k = 0; k < groups; ++k)
            for (int g = 0; g < G; ++g) sum += acc_smem[k * row_pad + c * G + g];
        p.partial[static_cast<long long>(blockIdx.x) * p.C + c] = sum;
    }
}

// dw[c] = sum over blocks, in float64 and in block order within 16 interleaved slices that
// are then added in slice order: the same bits for the same launch shape.
__global__ void __launch_bounds__(512) eqlin_rmsnorm_dw_kernel(const float* partial, float* dw, int C, int blocks) {
    __shared__ double part[16][33];
    ptx::grid_dependency_wait();
    const int c = blockIdx.x * 32 + threadIdx.x;
    double s = 0.0;
    if (c < C) {
#pragma unroll 16   // reads in flight: the launch is short, and bound by their latency
        for (int b = threadIdx.y; b < blocks; b += 16) s += partial[static_cast<long long>(b) * C + c];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < C) {
        for (int k = 1; k < 16; ++k) s += part[k][threadIdx.x];
        dw[c] = static_cast<float>(s);
    }
}

}  // namespace norm
}  // namespace eqlin
