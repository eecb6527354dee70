// eqlin_attn_f32.cuh -- attention in fp32 arithmetic on the CUDA cores, for calls of so few rows that tiles of 64
// would leave most SMs idle.
//
// One block of 256 threads (16 x 16) holds a tile of 16 rows and walks the other side in tiles of 64, copied
// asynchronously a tile ahead: one pass with a running maximum and sum per row.  A thread owns row ty and the 4
// columns (tx, tx + 16, ..) of the products, and the columns tx * 4 + 64 j of its row's accumulators.  What bounds
// it is latency: 256 tokens, one head of 64 features take 17 us forward and 29 us for all gradients, a chain of
// four tiles.  Copies fill with zeros past the ends, so rows of another sequence, whatever they hold, never enter
// a product.
#pragma once

#include "eqlin_attn.cuh"

namespace eqlin {
namespace attn {
namespace f32 {

constexpr int kN = 64;          // rows of a tile of the side that is walked
constexpr int kThreads = 256;
constexpr int kPS = kN + 4;     // row stride of the weights in shared memory

template <int DP>
struct Shape {
    static constexpr int M = 16;
    static constexpr int RS = DP + 4;                    // row stride of a feature tile (floats)
    static constexpr int OWN = M * RS, WALK = kN * RS, W = M * kPS;
    static constexpr int FWD_BYTES = (OWN + 4 * WALK + W) * 4;
    static constexpr int DKV_BYTES = (2 * OWN + 2 * (2 * WALK + 2 * kN) + 2 * W) * 4;
    static constexpr int DQ_BYTES = (2 * OWN + 4 * WALK + W) * 4;
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

// acc[b] += sum_d A[ty][d] B[tx + 16 b][d]
template <int DP>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx, float (&acc)[4]) {
    constexpr int RS = DP + 4;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        const float4 a = *reinterpret_cast<const float4*>(A + ty * RS + d);
        float4 b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const float4*>(B + (tx + 16 * i) * RS + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] = fmaf(a.x, b[j].x, acc[j]);
            acc[j] = fmaf(a.y, b[j].y, acc[j]);
            acc[j] = fmaf(a.z, b[j].z, acc[j]);
            acc[j] = fmaf(a.w, b[j].w, acc[j]);
        }
    }
}

// acc[4 j + e] += sum_c P[ty][c] B[c][tx * 4 + 64 j + e]; P rows have stride kPS.
template <int DP>
__device__ __forceinline__ void apply_tile(const float* P, const float* B, int ty, int tx, float (&acc)[DP / 16]) {
    constexpr int RS = DP + 4;
#pragma unroll 4
    for (int c = 0; c < kN; c += 4) {
        const float4 pr = *reinterpret_cast<const float4*>(P + ty * kPS + c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < DP / 64; ++j) {
                const float4 b = *reinterpret_cast<const float4*>(B + (c + k) * RS + tx * 4 + 64 * j);
                const float w = k == 0 ? pr.x : k == 1 ? pr.y : k == 2 ? pr.z : pr.w;
                acc[4 * j] = fmaf(w, b.x, acc[4 * j]);
                acc[4 * j + 1] = fmaf(w, b.y, acc[4 * j + 1]);
                acc[4 * j + 2] = fmaf(w, b.z, acc[4 * j + 2]);
                acc[4 * j + 3] = fmaf(w, b.w, acc[4 * j + 3]);
            }
    }
}

template <int DP>
__device__ __forceinline__ void store_rows(void* base, long long stride, long long row0, int n, int D, int head, int ty,
                                           int tx, const float (&acc)[DP / 16], float mul) {
    if (ty >= n) return;
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) {
        const int c = tx * 4 + 64 * j;
        if (c < D)
            *reinterpret_cast<float4*>(static_cast<float*>(base) + (row0 + ty) * stride +
                                       static_cast<long long>(head) * D + c) =
                make_float4(acc[4 * j] * mul, acc[4 * j + 1] * mul, acc[4 * j + 2] * mul,
                            acc[4 * j + 3] * mul);
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

template <int DP>
__global__ void __launch_bounds__(kThreads) eqlin_attn_fwd_f32_kernel(const Params p) {
    extern __shared__ __align__(16) float smem[];
    using S = Shape<DP>;
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
    float top = -INFINITY, sum = 0.f, acc[DP / 16] = {};
    for (int k = begin; k < end; ++k) {
        if (k + 1 < end) fetch(k + 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const float *sk = skv + (k & 1) * 2 * S::WALK, *sv = sk + S::WALK;
        float s[4] = {};
        dot_tile<DP>(sq, sk, ty, tx, s);
        const int last = p.causal ? r0 + ty - t.own.len + kr.len : kr.len - 1;
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = k * kN + tx + 16 * j;
            s[j] = col < kr.len && col <= last ? s[j] * c2 : -INFINITY;
            m = fmaxf(m, s[j]);
        }
        m = fmaxf(top, row_max(m));
        const float ref = m == -INFINITY ? 0.f : m;
        const float fade = exp2f(top - ref);   // 0 while top is -infinity
        top = m;
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] = exp2f(s[j] - ref);
            part += s[j];
            sp[ty * kPS + tx + 16 * j] = s[j];
        }
        sum = sum * fade + part;
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) acc[j] *= fade;
        __syncwarp();   // a row's 16 threads are lanes of one warp
        apply_tile<DP>(sp, sv, ty, tx, acc);
        __syncthreads();
    }
    cp_async_wait<0>();   // without keys the copy of Q is still on its way
    sum = row_sum(sum);
    const float mul = sum == 0.f ? 0.f : 1.f / sum;   // a row that sees no key
    const float lse = sum == 0.f ? -INFINITY : fmaf(top, kLn2, logf(sum));
    const long long at = static_cast<long long>(h) * p.q_rows + t.own.start + r0 + ty;
    if (tx == 0 && ty < n) {
        if (p.splits > 1) p.part_lse[static_cast<long long>(blockIdx.z) * p.heads * p.q_rows + at] = lse;
        else if (p.lse) p.lse[at] = lse;
    }
    if (p.splits > 1)   // rows of D floats, one head
        store_rows<DP>(p.part_o + (static_cast<long long>(blockIdx.z) * p.heads + h) * p.q_rows * p.D, p.D,
                          static_cast<long long>(t.own.start) + r0, n, p.D, 0, ty, tx, acc, mul);
    else
        store_rows<DP>(p.out, p.o_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h, ty, tx, acc, mul);
}

// dk and dv: a tile of keys walks the query rows that see it, for each query head of its group.
template <int DP>
__device__ __forceinline__ void dkv_tile(const Params& p, float* smem, int slot, int hk) {
    using S = Shape<DP>;
    constexpr int STAGE = 2 * S::WALK + 2 * kN;      // Q, dO, lse, delta
    float *sk = smem, *sv = sk + S::OWN, *walk = sv + S::OWN;
    float *sp = walk + 2 * STAGE, *sds = sp + S::W;
    const int group = p.heads / p.kv_heads;
    const Tile t = find_tile<S::M>(p.k_offsets, p.sequences, p.k_rows, slot);
    if (t.tile < 0) return;
    const Rows qr = other_rows(p, t, p.q_offsets, p.q_rows);
    const int r0 = t.tile * S::M, n = min(S::M, t.own.len - r0);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int begin = first_query(r0, qr.len, t.own.len, p.causal) / kN;
    const int per_head = max(0, (qr.len + kN - 1) / kN - begin), steps = per_head * group;
    auto fetch = [&](int u) {
        float* s = walk + (u & 1) * STAGE;
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
    if (steps > 0) fetch(0);
    cp_async_commit();
    const float c2 = p.scale * kLog2e;
    float dk[DP / 16] = {}, dv[DP / 16] = {};
    for (int u = 0; u < steps; ++u) {
        if (u + 1 < steps) fetch(u + 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const float *sq = walk + (u & 1) * STAGE, *sdo = sq + S::WALK, *slse = sdo + S::WALK, *sdelta = slse + kN;
        const int q0 = (begin + u % per_head) * kN;
        float s[4] = {}, dp[4] = {};   // rows are keys, columns are queries
        dot_tile<DP>(sk, sq, ty, tx, s);
        dot_tile<DP>(sv, sdo, ty, tx, dp);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = r0 + ty, query = q0 + tx + 16 * j;
            const bool vis = !p.causal || key <= query - qr.len + t.own.len;
            const float w = vis ? exp2f(s[j] * c2 - slse[tx + 16 * j]) : 0.f;
            sp[ty * kPS + tx + 16 * j] = w;
            sds[ty * kPS + tx + 16 * j] = vis ? w * (dp[j] - sdelta[tx + 16 * j]) : 0.f;
        }
        __syncwarp();
        apply_tile<DP>(sp, sdo, ty, tx, dv);
        apply_tile<DP>(sds, sq, ty, tx, dk);
        __syncthreads();
    }
    cp_async_wait<0>();   // without queries those of K and V
    store_rows<DP>(p.dv, p.dv_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk, ty, tx, dv, 1.f);
    store_rows<DP>(p.dk, p.dk_stride, static_cast<long long>(t.own.start) + r0, n, p.D, hk, ty, tx, dk, p.scale);
}

// dq: a tile of queries walks the keys that it sees.
template <int DP>
__device__ __forceinline__ void dq_tile(const Params& p, float* smem, int slot, int h) {
    using S = Shape<DP>;
    float *sq = smem, *sdo = sq + S::OWN, *walk = sdo + S::OWN, *sds = walk + 4 * S::WALK;
    const int hk = h / (p.heads / p.kv_heads);
    const Tile t = find_tile<S::M>(p.q_offsets, p.sequences, p.q_rows, slot);
    if (t.tile < 0) return;
    const Rows kr = other_rows(p, t, p.k_offsets, p.k_rows);
    const int r0 = t.tile * S::M, n = min(S::M, t.own.len - r0);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int steps = (keys_seen(r0 + n - 1, t.own.len, kr.len, p.causal) + kN - 1) / kN;
    auto fetch = [&](int k) {
        float* s = walk + (k & 1) * 2 * S::WALK;
        load_tile<DP, kN>(s, p.k, p.k_stride, static_cast<long long>(kr.start) + k * kN, kr.len - k * kN, p.D, hk);
        load_tile<DP, kN>(s + S::WALK, p.v, p.v_stride, static_cast<long long>(kr.start) + k * kN, kr.len - k * kN, p.D, hk);
    };
    load_tile<DP, S::M>(sq, p.q, p.q_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h);
    load_tile<DP, S::M>(sdo, p.dout, p.do_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h);
    if (steps > 0) fetch(0);
    cp_async_commit();
    const float c2 = p.scale * kLog2e;
    float dq[DP / 16] = {};
    const long long at = static_cast<long long>(h) * p.q_rows + t.own.start + r0 + ty;
    const float lse2 = ty < n ? p.lse[at] * kLog2e : 0.f;
    const float delta = ty < n ? p.delta[at] : 0.f;
    for (int k = 0; k < steps; ++k) {
        if (k + 1 < steps) fetch(k + 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const float *sk = walk + (k & 1) * 2 * S::WALK, *sv = sk + S::WALK;
        float s[4] = {}, dp[4] = {};
        dot_tile<DP>(sq, sk, ty, tx, s);
        dot_tile<DP>(sdo, sv, ty, tx, dp);
        const int last = p.causal ? r0 + ty - t.own.len + kr.len : kr.len - 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = k * kN + tx + 16 * j;
            const bool vis = col < kr.len && col <= last;
            sds[ty * kPS + tx + 16 * j] = vis ? exp2f(s[j] * c2 - lse2) * (dp[j] - delta) : 0.f;
        }
        __syncwarp();
        apply_tile<DP>(sds, sk, ty, tx, dq);
        __syncthreads();
    }
    cp_async_wait<0>();
    store_rows<DP>(p.dq, p.dq_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h, ty, tx, dq, p.scale);
}

// All gradients in one launch: the first k_blocks blocks take tiles of keys, the rest tiles of queries (heads
// fastest).  Neither side waits for the other, and small problems fill more SMs.
template <int DP>
__global__ void __launch_bounds__(kThreads) eqlin_attn_bwd_f32_kernel(const Params p, unsigned k_blocks) {
    extern __shared__ __align__(16) float smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    if (blockIdx.x < k_blocks) {
        dkv_tile<DP>(p, smem, blockIdx.x / p.kv_heads, blockIdx.x % p.kv_heads);
    } else {
        const unsigned b = blockIdx.x - k_blocks;
        dq_tile<DP>(p, smem, b / p.heads, b % p.heads);
    }
}

}  // namespace f32
}  // namespace attn
}  // namespace eqlin
