// eqlin_attn_f32.cuh -- attention in fp32 arithmetic on the CUDA cores.
//
// One block of 256 threads (16 x 16) holds a tile of 16 R rows and walks the other side in tiles of 64, copied
// asynchronously a tile ahead where shared memory allows: one pass with a running maximum and sum per row.  A
// thread owns R rows (ty * R ..) and 4 columns (tx, tx + 16, ..) of the products, and the columns tx * 4 + 64 j
// of its rows' accumulators.  R = 4 is bound by the FMA pipes (64 FMAs for 8 vector loads from shared memory);
// R = 1 gives four times the blocks where R = 4 would leave SMs idle.  Copies fill with zeros past the ends, so
// rows of another sequence, whatever they hold, never enter a product.
#pragma once

#include "eqlin_attn.cuh"

namespace eqlin {
namespace attn {
namespace f32 {

constexpr int kN = 64;          // rows of a tile of the side that is walked
constexpr int kThreads = 256;
constexpr int kPS = kN + 4;     // row stride of the weights in shared memory

template <int DP, int R>
struct Shape {
    static constexpr int M = 16 * R;
    static constexpr int RS = DP + 4;                    // row stride of a feature tile (floats)
    static constexpr int OWN = M * RS, WALK = kN * RS, W = M * kPS;
    static constexpr int STAGES = R == 1 ? 2 : 1;        // of the gradients' walked tiles; the forward has 2
    static constexpr int FWD_BYTES = (OWN + 4 * WALK + W) * 4;
    static constexpr int DKV_BYTES = (2 * OWN + STAGES * (2 * WALK + 2 * kN) + 2 * W) * 4;
    static constexpr int DQ_BYTES = (2 * OWN + STAGES * 2 * WALK + W) * 4;
};

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(take ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows [0, ROWS) of a tile into shared memory; rows >= n and columns >= D as zeros.
template <int DP, int ROWS>
__device__ __forceinline__ void load_tile(float* s, const void* base, long long stride, long long row0, int n, int D,
                                          int head) {
    constexpr int STEP = kThreads / (DP / 4);
    const int c = threadIdx.x % (DP / 4) * 4, r0 = threadIdx.x / (DP / 4);
    const float* g = static_cast<const float*>(base) + static_cast<long long>(head) * D + c;
#pragma unroll
    for (int k = 0; k < (ROWS + STEP - 1) / STEP; ++k) {
        const int r = r0 + k * STEP;
        if (ROWS % STEP && r >= ROWS) break;
        const bool take = r < n && c < D;
        cp_async16(s + r * (DP + 4) + c, take ? g + (row0 + r) * stride : static_cast<const float*>(base), take);
    }
}

// acc[a][b] += sum_d A[ty * R + a][d] B[tx + 16 b][d]
template <int DP, int R>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx, float (&acc)[R][4]) {
    constexpr int RS = DP + 4;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float4 a[R], b[4];
#pragma unroll
        for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty * R + i) * RS + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const float4*>(B + (tx + 16 * i) * RS + d);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
                acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
                acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
                acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
            }
    }
}

// acc[a][4 j + e] += sum_c P[ty * R + a][c] B[c][tx * 4 + 64 j + e]; P rows have stride kPS.
template <int DP, int R>
__device__ __forceinline__ void apply_tile(const float* P, const float* B, int ty, int tx, float (&acc)[R][DP / 16]) {
    constexpr int RS = DP + 4;
#pragma unroll 4
    for (int c = 0; c < kN; c += 4) {
        float4 pr[R];
#pragma unroll
        for (int i = 0; i < R; ++i) pr[i] = *reinterpret_cast<const float4*>(P + (ty * R + i) * kPS + c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < DP / 64; ++j) {
                const float4 b = *reinterpret_cast<const float4*>(B + (c + k) * RS + tx * 4 + 64 * j);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float w = k == 0 ? pr[i].x : k == 1 ? pr[i].y : k == 2 ? pr[i].z : pr[i].w;
                    acc[i][4 * j] = fmaf(w, b.x, acc[i][4 * j]);
                    acc[i][4 * j + 1] = fmaf(w, b.y, acc[i][4 * j + 1]);
                    acc[i][4 * j + 2] = fmaf(w, b.z, acc[i][4 * j + 2]);
                    acc[i][4 * j + 3] = fmaf(w, b.w, acc[i][4 * j + 3]);
                }
            }
    }
}

template <int DP, int R>
__device__ __forceinline__ void store_rows(void* base, long long stride, long long row0, int n, int D, int head, int ty,
                                           int tx, const float (&acc)[R][DP / 16], const float (&mul)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (ty * R + i >= n) continue;
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
            const int c = tx * 4 + 64 * j;
            if (c < D)
                *reinterpret_cast<float4*>(static_cast<float*>(base) + (row0 + ty * R + i) * stride +
                                           static_cast<long long>(head) * D + c) =
                    make_float4(acc[i][4 * j] * mul[i], acc[i][4 * j + 1] * mul[i], acc[i][4 * j + 2] * mul[i],
                                acc[i][4 * j + 3] * mul[i]);
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

template <int DP, int R>
__global__ void __launch_bounds__(kThreads) eqlin_attn_fwd_f32_kernel(const Params p) {
    extern __shared__ __align__(16) float smem[];
    using S = Shape<DP, R>;
    float *sq = smem, *skv = sq + S::OWN, *sp = skv + 4 * S::WALK;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int h = blockIdx.y, hk = h / (p.heads / p.kv_heads);
    const Tile t = find_tile<S::M>(p.q_offsets, p.sequences, p.q_rows, blockIdx.x);
    if (t.tile < 0) return;
    const Rows kr = other_rows(p, t, p.k_offsets, p.k_rows);
    const int r0 = t.tile * S::M, n = min(S::M, t.own.len - r0);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int seen = keys_seen(r0 + n - 1, t.own.len, kr.len, p.causal);
    // this slice's tiles of keys (all of them unless the keys are split)
    const int tiles = (seen + kN - 1) / kN;
    const int begin = static_cast<int>(static_cast<long long>(tiles) * blockIdx.z / p.splits);
    const int end = static_cast<int>(static_cast<long long>(tiles) * (blockIdx.z + 1) / p.splits);
    auto fetch = [&](int k) {
        float* s = skv + (k & 1) * 2 * S::WALK;
        const int kn = kr.len - k * kN;
        load_tile<DP, kN>(s, p.k, p.k_stride, static_cast<long long>(kr.start) + k * kN, kn, p.D, hk);
        load_tile<DP, kN>(s + S::WALK, p.v, p.v_stride, static_cast<long long>(kr.start) + k * kN, kn, p.D, hk);
    };
    load_tile<DP, S::M>(sq, p.q, p.q_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h);
    if (begin < end) fetch(begin);
    cp_async_commit();
    const float c2 = p.scale * kLog2e;
    float top[R], sum[R], acc[R][DP / 16];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        top[i] = -INFINITY;
        sum[i] = 0.f;
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) acc[i][j] = 0.f;
    }
    for (int k = begin; k < end; ++k) {
        if (k + 1 < end) fetch(k + 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const float *sk = skv + (k & 1) * 2 * S::WALK, *sv = sk + S::WALK;
        float s[R][4] = {};
        dot_tile<DP, R>(sq, sk, ty, tx, s);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int last = p.causal ? r0 + ty * R + i + kr.len - t.own.len : kr.len - 1;
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = k * kN + tx + 16 * j;
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
                sp[(ty * R + i) * kPS + tx + 16 * j] = s[i][j];
            }
            sum[i] = sum[i] * fade + part;
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) acc[i][j] *= fade;
        }
        __syncwarp();   // a row's 16 threads are lanes of one warp
        apply_tile<DP, R>(sp, sv, ty, tx, acc);
        __syncthreads();
    }
    float mul[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        sum[i] = row_sum(sum[i]);
        mul[i] = sum[i] == 0.f ? 0.f : 1.f / sum[i];   // a row that sees no key
        const float lse = sum[i] == 0.f ? -INFINITY : fmaf(top[i], kLn2, logf(sum[i]));
        const long long at = static_cast<long long>(h) * p.q_rows + t.own.start + r0 + ty * R + i;
        if (tx != 0 || ty * R + i >= n) continue;
        if (p.splits > 1) p.part_lse[static_cast<long long>(blockIdx.z) * p.heads * p.q_rows + at] = lse;
        else if (p.lse) p.lse[at] = lse;
    }
    if (p.splits > 1)   // rows of D floats, one head
        store_rows<DP, R>(p.part_o + (static_cast<long long>(blockIdx.z) * p.heads + h) * p.q_rows * p.D, p.D,
                          static_cast<long long>(t.own.start) + r0, n, p.D, 0, ty, tx, acc, mul);
    else
        store_rows<DP, R>(p.out, p.o_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h, ty, tx, acc, mul);
}

// dk and dv: a tile of keys walks the query rows that see it, for each query head of its group.
template <int DP, int R>
__device__ __forceinline__ void dkv_tile(const Params& p, float* smem, int slot, int hk) {
    using S = Shape<DP, R>;
    constexpr int STAGE = 2 * S::WALK + 2 * kN;      // Q, dO, lse, delta
    float *sk = smem, *sv = sk + S::OWN, *walk = sv + S::OWN;
    float *sp = walk + S::STAGES * STAGE, *sds = sp + S::W;
    const int group = p.heads / p.kv_heads;
    const Tile t = find_tile<S::M>(p.k_offsets, p.sequences, p.k_rows, slot);
    if (t.tile < 0) return;
    const Rows qr = other_rows(p, t, p.q_offsets, p.q_rows);
    const int r0 = t.tile * S::M, n = min(S::M, t.own.len - r0);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int begin = first_query(r0, qr.len, t.own.len, p.causal) / kN;
    const int per_head = max(0, (qr.len + kN - 1) / kN - begin), steps = per_head * group;
    auto fetch = [&](int u) {
        float* s = walk + (u % S::STAGES) * STAGE;
        const int h = hk * group + u / per_head, q0 = (begin + u % per_head) * kN, qn = qr.len - q0;
        load_tile<DP, kN>(s, p.q, p.q_stride, static_cast<long long>(qr.start) + q0, qn, p.D, h);
        load_tile<DP, kN>(s + S::WALK, p.dout, p.do_stride, static_cast<long long>(qr.start) + q0, qn, p.D, h);
        if (threadIdx.x < kN) {
            const long long at = static_cast<long long>(h) * p.q_rows + qr.start + q0 + threadIdx.x;
            const float l = static_cast<int>(threadIdx.x) < qn ? p.lse[at] : -INFINITY;
            s[2 * S::WALK + threadIdx.x] = l == -INFINITY ? INFINITY : l * kLog2e;   // weights of zero
            s[2 * S::WALK + kN + threadIdx.x] = static_cast<int>(threadIdx.x) < qn ? p.delta[at] : 0.f;
        }
    };
    load_tile<DP, S::M>(sk, p.k, p.k_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk);
    load_tile<DP, S::M>(sv, p.v, p.v_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk);
    if (S::STAGES == 2 && steps > 0) fetch(0);
    cp_async_commit();
    const float c2 = p.scale * kLog2e;
    float dk[R][DP / 16] = {}, dv[R][DP / 16] = {};
    for (int u = 0; u < steps; ++u) {
        if (S::STAGES == 1) fetch(u);
        else if (u + 1 < steps) fetch(u + 1);
        cp_async_commit();
        cp_async_wait<S::STAGES - 1>();
        __syncthreads();
        const float *sq = walk + (u % S::STAGES) * STAGE, *sdo = sq + S::WALK, *slse = sdo + S::WALK, *sdelta = slse + kN;
        const int q0 = (begin + u % per_head) * kN;
        float s[R][4] = {}, dp[R][4] = {};   // rows are keys, columns are queries
        dot_tile<DP, R>(sk, sq, ty, tx, s);
        dot_tile<DP, R>(sv, sdo, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = r0 + ty * R + i, query = q0 + tx + 16 * j;
                const bool vis = !p.causal || key <= query + t.own.len - qr.len;
                const float w = vis ? exp2f(s[i][j] * c2 - slse[tx + 16 * j]) : 0.f;
                sp[(ty * R + i) * kPS + tx + 16 * j] = w;
                sds[(ty * R + i) * kPS + tx + 16 * j] = vis ? w * (dp[i][j] - sdelta[tx + 16 * j]) : 0.f;
            }
        __syncwarp();
        apply_tile<DP, R>(sp, sdo, ty, tx, dv);
        apply_tile<DP, R>(sds, sq, ty, tx, dk);
        __syncthreads();
    }
    float one[R], sc[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        one[i] = 1.f;
        sc[i] = p.scale;
    }
    store_rows<DP, R>(p.dv, p.dv_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk, ty, tx, dv, one);
    store_rows<DP, R>(p.dk, p.dk_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk, ty, tx, dk, sc);
}

// dq: a tile of queries walks the keys that it sees.
template <int DP, int R>
__device__ __forceinline__ void dq_tile(const Params& p, float* smem, int slot, int h) {
    using S = Shape<DP, R>;
    float *sq = smem, *sdo = sq + S::OWN, *walk = sdo + S::OWN, *sds = walk + S::STAGES * 2 * S::WALK;
    const int hk = h / (p.heads / p.kv_heads);
    const Tile t = find_tile<S::M>(p.q_offsets, p.sequences, p.q_rows, slot);
    if (t.tile < 0) return;
    const Rows kr = other_rows(p, t, p.k_offsets, p.k_rows);
    const int r0 = t.tile * S::M, n = min(S::M, t.own.len - r0);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int steps = (keys_seen(r0 + n - 1, t.own.len, kr.len, p.causal) + kN - 1) / kN;
    auto fetch = [&](int k) {
        float* s = walk + (k % S::STAGES) * 2 * S::WALK;
        load_tile<DP, kN>(s, p.k, p.k_stride, static_cast<long long>(kr.start) + k * kN, kr.len - k * kN, p.D, hk);
        load_tile<DP, kN>(s + S::WALK, p.v, p.v_stride, static_cast<long long>(kr.start) + k * kN, kr.len - k * kN, p.D, hk);
    };
    load_tile<DP, S::M>(sq, p.q, p.q_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h);
    load_tile<DP, S::M>(sdo, p.dout, p.do_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h);
    if (S::STAGES == 2 && steps > 0) fetch(0);
    cp_async_commit();
    const float c2 = p.scale * kLog2e;
    float lse2[R], delta[R], dq[R][DP / 16] = {};
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const long long at = static_cast<long long>(h) * p.q_rows + t.own.start + r0 + ty * R + i;
        lse2[i] = ty * R + i < n ? p.lse[at] * kLog2e : 0.f;
        delta[i] = ty * R + i < n ? p.delta[at] : 0.f;
    }
    for (int k = 0; k < steps; ++k) {
        if (S::STAGES == 1) fetch(k);
        else if (k + 1 < steps) fetch(k + 1);
        cp_async_commit();
        cp_async_wait<S::STAGES - 1>();
        __syncthreads();
        const float *sk = walk + (k % S::STAGES) * 2 * S::WALK, *sv = sk + S::WALK;
        float s[R][4] = {}, dp[R][4] = {};
        dot_tile<DP, R>(sq, sk, ty, tx, s);
        dot_tile<DP, R>(sdo, sv, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int last = p.causal ? r0 + ty * R + i + kr.len - t.own.len : kr.len - 1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = k * kN + tx + 16 * j;
                const bool vis = col < kr.len && col <= last;
                sds[(ty * R + i) * kPS + tx + 16 * j] = vis ? exp2f(s[i][j] * c2 - lse2[i]) * (dp[i][j] - delta[i]) : 0.f;
            }
        }
        __syncwarp();
        apply_tile<DP, R>(sds, sk, ty, tx, dq);
        __syncthreads();
    }
    float sc[R];
#pragma unroll
    for (int i = 0; i < R; ++i) sc[i] = p.scale;
    store_rows<DP, R>(p.dq, p.dq_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h, ty, tx, dq, sc);
}

// All gradients in one launch: the first k_blocks blocks take tiles of keys, the rest tiles of queries (heads
// fastest).  Neither side waits for the other, and small problems fill more SMs.
template <int DP, int R>
__global__ void __launch_bounds__(kThreads) eqlin_attn_bwd_f32_kernel(const Params p, unsigned k_blocks) {
    extern __shared__ __align__(16) float smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    if (blockIdx.x < k_blocks) {
        dkv_tile<DP, R>(p, smem, blockIdx.x / p.kv_heads, blockIdx.x % p.kv_heads);
    } else {
        const unsigned b = blockIdx.x - k_blocks;
        dq_tile<DP, R>(p, smem, b / p.heads, b % p.heads);
    }
}

}  // namespace f32
}  // namespace attn
}  // namespace eqlin
