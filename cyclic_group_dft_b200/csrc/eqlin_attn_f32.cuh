// eqlin_attn_f32.cuh -- attention in fp32 arithmetic on the CUDA cores.
//
// One block of 256 threads (16 x 16) holds a tile of 64 rows and walks the other side in tiles of
// 64: one pass with a running maximum and sum per row.  A thread owns 4 rows (ty * 4 ..) and 4
// columns (tx, tx + 16, ..) of the 64 x 64 products, and the columns tx * 4 + 64 j of its rows'
// accumulators.  Tiles are zero-filled past the ends, so rows of another sequence, whatever they
// hold, never enter a product.
#pragma once

#include "eqlin_attn.cuh"

namespace eqlin {
namespace attn {
namespace f32 {

constexpr int kM = 64;          // rows of a tile, both sides
constexpr int kThreads = 256;
constexpr int kPS = kM + 4;     // row stride of the 64 x 64 tiles in shared memory

template <int DP>
struct Shape {
    static constexpr int RS = DP + 4;                    // row stride of a feature tile (floats)
    static constexpr int TILE = kM * RS;
    static constexpr int FWD_BYTES = (3 * TILE + kM * kPS) * 4;
    static constexpr int DKV_BYTES = (4 * TILE + 2 * kM * kPS + 2 * kM) * 4;
    static constexpr int DQ_BYTES = (4 * TILE + kM * kPS) * 4;
};

// Rows [0, 64) of a tile into shared memory as fp32; rows >= n and columns >= D as zeros.
template <class T, int DP>
__device__ __forceinline__ void load_tile(float* s, const void* base, long long stride, long long row0, int n, int D,
                                          int head) {
    constexpr int VEC = 16 / sizeof(T);
    using V = Vec<T, VEC>;
    for (int i = threadIdx.x; i < kM * (DP / VEC); i += kThreads) {
        const int r = i / (DP / VEC), c = (i - r * (DP / VEC)) * VEC;
        float v[VEC];
        typename V::Raw raw = typename V::Raw{};
        if (r < n && c < D)
            raw = V::load(static_cast<const T*>(base) + (row0 + r) * stride + static_cast<long long>(head) * D + c);
        V::unpack(raw, v);
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
            *reinterpret_cast<float4*>(s + r * Shape<DP>::RS + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    }
}

// acc[a][b] += sum_d A[ty * 4 + a][d] B[tx + 16 b][d]
template <int DP>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx, float (&acc)[4][4]) {
    constexpr int RS = Shape<DP>::RS;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4*>(A + (ty * 4 + i) * RS + d);
            b[i] = *reinterpret_cast<const float4*>(B + (tx + 16 * i) * RS + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
                acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
                acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
                acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
            }
    }
}

// acc[a][4 j + e] += sum_{c < n} P[ty * 4 + a][c] B[c][tx * 4 + 64 j + e]; P rows have stride kPS.
template <int DP>
__device__ __forceinline__ void apply_tile(const float* P, const float* B, int ty, int tx, int n,
                                           float (&acc)[4][DP / 16]) {
    constexpr int RS = Shape<DP>::RS;
    constexpr int J = DP / 64 > 0 ? DP / 64 : 1;
    const bool on = DP >= 64 || tx * 4 < DP;
    if (!on) return;
#pragma unroll 2
    for (int c = 0; c < n; c += 4) {
        float4 pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4*>(P + (ty * 4 + i) * kPS + c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float4 b = *reinterpret_cast<const float4*>(B + (c + k) * RS + tx * 4 + 64 * j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = k == 0 ? pr[i].x : k == 1 ? pr[i].y : k == 2 ? pr[i].z : pr[i].w;
                    acc[i][4 * j] = fmaf(w, b.x, acc[i][4 * j]);
                    acc[i][4 * j + 1] = fmaf(w, b.y, acc[i][4 * j + 1]);
                    acc[i][4 * j + 2] = fmaf(w, b.z, acc[i][4 * j + 2]);
                    acc[i][4 * j + 3] = fmaf(w, b.w, acc[i][4 * j + 3]);
                }
            }
    }
}

template <class T, int DP>
__device__ __forceinline__ void store_rows(void* base, long long stride, long long row0, int n, int D, int head, int ty,
                                           int tx, const float (&acc)[4][DP / 16], const float (&mul)[4]) {
    using V = Vec<T, 4>;
    constexpr int J = DP / 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (ty * 4 + i >= n) continue;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = tx * 4 + 64 * j;
            if (c >= D) continue;
            const float v[4] = {acc[i][4 * j] * mul[i], acc[i][4 * j + 1] * mul[i], acc[i][4 * j + 2] * mul[i],
                                acc[i][4 * j + 3] * mul[i]};
            V::store(static_cast<T*>(base) + (row0 + ty * 4 + i) * stride + static_cast<long long>(head) * D + c,
                     V::pack(v));
        }
    }
}

// sum / max over the 16 threads that share a row (lanes of one half warp)
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <class T, int DP>
__global__ void __launch_bounds__(kThreads) eqlin_attn_fwd_f32_kernel(const Params p) {
    extern __shared__ __align__(16) float smem[];
    constexpr int TILE = Shape<DP>::TILE;
    float *sq = smem, *sk = sq + TILE, *sv = sk + TILE, *sp = sv + TILE;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int h = blockIdx.y, hk = h / (p.heads / p.kv_heads);
    const Tile t = find_tile<kM>(p.q_offsets, p.sequences, p.q_rows, blockIdx.x);
    if (t.tile < 0) return;
    const Rows kr = sequence_rows(p.k_offsets, t.b, p.k_rows);
    const int r0 = t.tile * kM, n = min(kM, t.own.len - r0);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int seen = keys_seen(r0 + n - 1, t.own.len, kr.len, p.causal);
    // this slice's tiles of keys (all of them unless the keys are split)
    const int tiles = (seen + kM - 1) / kM;
    const int begin = static_cast<int>(static_cast<long long>(tiles) * blockIdx.z / p.splits) * kM;
    const int end = min(seen, static_cast<int>(static_cast<long long>(tiles) * (blockIdx.z + 1) / p.splits) * kM);
    load_tile<T, DP>(sq, p.q, p.q_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h);
    const float c2 = p.scale * kLog2e;
    float top[4], sum[4], acc[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        top[i] = -INFINITY;
        sum[i] = 0.f;
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) acc[i][j] = 0.f;
    }
    for (int k0 = begin; k0 < end; k0 += kM) {
        const int kn = min(kM, kr.len - k0);
        __syncthreads();
        load_tile<T, DP>(sk, p.k, p.k_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk);
        load_tile<T, DP>(sv, p.v, p.v_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk);
        __syncthreads();
        float s[4][4] = {};
        dot_tile<DP>(sq, sk, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int last = p.causal ? r0 + ty * 4 + i + kr.len - t.own.len : kr.len - 1;
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = k0 + tx + 16 * j;
                s[i][j] = col < kr.len && col <= last ? s[i][j] * c2 : -INFINITY;
                m = fmaxf(m, s[i][j]);
            }
            m = fmaxf(top[i], row_max(m));
            const float ref = m == -INFINITY ? 0.f : m;
            const float fade = exp2f(top[i] - ref);   // 0 while top is -infinity
            top[i] = m;
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - ref);
                part += s[i][j];
                sp[(ty * 4 + i) * kPS + tx + 16 * j] = s[i][j];
            }
            sum[i] = sum[i] * fade + part;
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) acc[i][j] *= fade;
        }
        __syncwarp();   // a row's 16 threads are lanes of one warp
        apply_tile<DP>(sp, sv, ty, tx, kM, acc);
    }
    float mul[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum[i] = row_sum(sum[i]);
        mul[i] = sum[i] > 0.f || sum[i] != sum[i] ? 1.f / sum[i] : 0.f;
        const float lse = sum[i] == 0.f ? -INFINITY : fmaf(top[i], kLn2, logf(sum[i]));
        const long long at = static_cast<long long>(h) * p.q_rows + t.own.start + r0 + ty * 4 + i;
        if (tx != 0 || ty * 4 + i >= n) continue;
        if (p.splits > 1) p.part_lse[static_cast<long long>(blockIdx.z) * p.heads * p.q_rows + at] = lse;
        else if (p.lse) p.lse[at] = lse;
    }
    if (p.splits > 1)   // rows of D floats, one head
        store_rows<float, DP>(p.part_o + (static_cast<long long>(blockIdx.z) * p.heads + h) * p.q_rows * p.D, p.D,
                              static_cast<long long>(t.own.start) + r0, n, p.D, 0, ty, tx, acc, mul);
    else
        store_rows<T, DP>(p.out, p.o_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h, ty, tx, acc, mul);
}

// dk and dv: a tile of 64 keys walks the query rows that see it, for each query head of its group.
template <class T, int DP>
__global__ void __launch_bounds__(kThreads) eqlin_attn_dkv_f32_kernel(const Params p) {
    extern __shared__ __align__(16) float smem[];
    constexpr int TILE = Shape<DP>::TILE;
    float *sk = smem, *sv = sk + TILE, *sq = sv + TILE, *sdo = sq + TILE;
    float *sp = sdo + TILE, *sds = sp + kM * kPS, *slse = sds + kM * kPS, *sdelta = slse + kM;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int hk = blockIdx.y, group = p.heads / p.kv_heads;
    const Tile t = find_tile<kM>(p.k_offsets, p.sequences, p.k_rows, blockIdx.x);
    if (t.tile < 0) return;
    const Rows qr = sequence_rows(p.q_offsets, t.b, p.q_rows);
    const int r0 = t.tile * kM, n = min(kM, t.own.len - r0);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    load_tile<T, DP>(sk, p.k, p.k_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk);
    load_tile<T, DP>(sv, p.v, p.v_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk);
    const float c2 = p.scale * kLog2e;
    float dk[4][DP / 16] = {}, dv[4][DP / 16] = {};
    const int begin = first_query(r0, qr.len, t.own.len, p.causal) / kM * kM;
    for (int hi = 0; hi < group; ++hi) {
        const int h = hk * group + hi;
        for (int q0 = begin; q0 < qr.len; q0 += kM) {
            const int qn = min(kM, qr.len - q0);
            __syncthreads();
            load_tile<T, DP>(sq, p.q, p.q_stride, static_cast<long long>(qr.start) + q0, qn, p.D, h);
            load_tile<T, DP>(sdo, p.dout, p.do_stride, static_cast<long long>(qr.start) + q0, qn, p.D, h);
            if (threadIdx.x < kM) {
                const long long at = static_cast<long long>(h) * p.q_rows + qr.start + q0 + threadIdx.x;
                slse[threadIdx.x] = threadIdx.x < qn ? p.lse[at] * kLog2e : 0.f;
                sdelta[threadIdx.x] = threadIdx.x < qn ? p.delta[at] : 0.f;
            }
            __syncthreads();
            float s[4][4] = {}, dp[4][4] = {};   // rows are keys, columns are queries
            dot_tile<DP>(sk, sq, ty, tx, s);
            dot_tile<DP>(sv, sdo, ty, tx, dp);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = r0 + ty * 4 + i, query = q0 + tx + 16 * j;
                    const bool vis = query < qr.len && key < t.own.len &&
                                     (!p.causal || key <= query + t.own.len - qr.len);
                    const float w = vis ? exp2f(s[i][j] * c2 - slse[tx + 16 * j]) : 0.f;
                    sp[(ty * 4 + i) * kPS + tx + 16 * j] = w;
                    sds[(ty * 4 + i) * kPS + tx + 16 * j] = vis ? w * (dp[i][j] - sdelta[tx + 16 * j]) : 0.f;
                }
            __syncwarp();
            apply_tile<DP>(sp, sdo, ty, tx, kM, dv);
            apply_tile<DP>(sds, sq, ty, tx, kM, dk);
        }
    }
    const float one[4] = {1.f, 1.f, 1.f, 1.f};
    const float sc[4] = {p.scale, p.scale, p.scale, p.scale};
    store_rows<T, DP>(p.dv, p.dv_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk, ty, tx, dv, one);
    store_rows<T, DP>(p.dk, p.dk_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk, ty, tx, dk, sc);
}

// dq: a tile of 64 queries walks the keys that it sees.
template <class T, int DP>
__global__ void __launch_bounds__(kThreads) eqlin_attn_dq_f32_kernel(const Params p) {
    extern __shared__ __align__(16) float smem[];
    constexpr int TILE = Shape<DP>::TILE;
    float *sq = smem, *sdo = sq + TILE, *sk = sdo + TILE, *sv = sk + TILE, *sds = sv + TILE;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int h = blockIdx.y, hk = h / (p.heads / p.kv_heads);
    const Tile t = find_tile<kM>(p.q_offsets, p.sequences, p.q_rows, blockIdx.x);
    if (t.tile < 0) return;
    const Rows kr = sequence_rows(p.k_offsets, t.b, p.k_rows);
    const int r0 = t.tile * kM, n = min(kM, t.own.len - r0);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int seen = keys_seen(r0 + n - 1, t.own.len, kr.len, p.causal);
    load_tile<T, DP>(sq, p.q, p.q_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h);
    load_tile<T, DP>(sdo, p.dout, p.do_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h);
    const float c2 = p.scale * kLog2e;
    float lse2[4], delta[4], dq[4][DP / 16] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long at = static_cast<long long>(h) * p.q_rows + t.own.start + r0 + ty * 4 + i;
        lse2[i] = ty * 4 + i < n ? p.lse[at] * kLog2e : 0.f;
        delta[i] = ty * 4 + i < n ? p.delta[at] : 0.f;
    }
    for (int k0 = 0; k0 < seen; k0 += kM) {
        const int kn = min(kM, kr.len - k0);
        __syncthreads();
        load_tile<T, DP>(sk, p.k, p.k_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk);
        load_tile<T, DP>(sv, p.v, p.v_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk);
        __syncthreads();
        float s[4][4] = {}, dp[4][4] = {};
        dot_tile<DP>(sq, sk, ty, tx, s);
        dot_tile<DP>(sdo, sv, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int last = p.causal ? r0 + ty * 4 + i + kr.len - t.own.len : kr.len - 1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = k0 + tx + 16 * j;
                const bool vis = col < kr.len && col <= last;
                sds[(ty * 4 + i) * kPS + tx + 16 * j] =
                    vis ? exp2f(s[i][j] * c2 - lse2[i]) * (dp[i][j] - delta[i]) : 0.f;
            }
        }
        __syncwarp();
        apply_tile<DP>(sds, sk, ty, tx, kM, dq);
    }
    const float sc[4] = {p.scale, p.scale, p.scale, p.scale};
    store_rows<T, DP>(p.dq, p.dq_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h, ty, tx, dq, sc);
}

}  // namespace f32
}  // namespace attn
}  // namespace eqlin
