// eqlin_attn_mma.cuh -- 16-bit attention where a 128-row tensor-core tile would be mostly empty: short
// sequences (windows of a few dozen tokens) and few queries over many keys.  Both are bound by memory,
// not by the tensor cores, and use 16-row warp products (mma.sync m16n8k16) whose scores and outputs
// stay in registers.
//
// Tiles in shared memory are rows of DP features; the 16-byte chunk c of row r lies at chunk
// c ^ (r & 7), so that ldmatrix reads eight rows without bank conflicts.  Rows past a sequence's end
// are filled with zeros by the copy itself.
#pragma once

#include "eqlin_attn.cuh"

namespace eqlin {
namespace attn {
namespace mma {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (Io16<T>::kUmmaFormat == 1)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int DP>
__device__ __forceinline__ uint32_t at(uint32_t tile, int row, int chunk) {
    return tile + row * (DP * 2) + ((chunk ^ (row & 7)) << 4);
}
// the four lanes of a row pair
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
    return v + __shfl_xor_sync(0xFFFFFFFFu, v, 2);
}

// acc[n8 tile] (16 rows of A x NT * 8 rows of B) += A B^T over the features, A and B row tiles.
template <class T, int DP, int NT>
__device__ __forceinline__ void rows_by_rows(float (&acc)[NT][4], uint32_t a_tile, uint32_t b_tile, int steps, int lane) {
    for (int ks = 0; ks < steps; ++ks) {
        uint32_t a[4];
        ldm4(a, at<DP>(a_tile, lane & 15, ks * 2 + (lane >> 4)));
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldm4(b, at<DP>(b_tile, n * 8 + (lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)));
            mma16816<T>(acc[n], a, b[0], b[1]);
            mma16816<T>(acc[n + 1], a, b[2], b[3]);
        }
    }
}
// o[feature tile] += P B: P = 16 rows x NT * 8 from accumulators rounded to T, B a row tile.
template <class T, int DP, int NT>
__device__ __forceinline__ void weights_by_rows(float (&o)[DP / 8][4], const float (&w)[NT][4], uint32_t b_tile, int D,
                                                int lane) {
#pragma unroll
    for (int kb = 0; kb < NT / 2; ++kb) {
        const uint32_t a[4] = {Io16<T>::pack(w[2 * kb][0], w[2 * kb][1]), Io16<T>::pack(w[2 * kb][2], w[2 * kb][3]),
                               Io16<T>::pack(w[2 * kb + 1][0], w[2 * kb + 1][1]),
                               Io16<T>::pack(w[2 * kb + 1][2], w[2 * kb + 1][3])};
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
            if (d * 16 >= D) break;
            uint32_t b[4];
            ldm4t(b, at<DP>(b_tile, kb * 16 + (lane & 15), d * 2 + (lane >> 4)));
            mma16816<T>(o[2 * d], a, b[0], b[1]);
            mma16816<T>(o[2 * d + 1], a, b[2], b[3]);
        }
    }
}

// Running softmax of 16 rows x NT * 8 keys: masks keys >= last[i] (relative to this tile) of row i of
// the pair, turns s into weights, moves the maximum and scales o and sum.
template <int NT, int DT>
__device__ __forceinline__ void softmax_step(float (&s)[NT][4], float (&o)[DT][4], float (&top)[2], float (&sum)[2],
                                             const int (&last)[2], float c2, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float m = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = n * 8 + (lane & 3) * 2 + e;
                s[n][2 * i + e] = col < last[i] ? s[n][2 * i + e] : -INFINITY;
                m = fmaxf(m, s[n][2 * i + e]);
            }
        m = fmaxf(top[i], quad_max(m));
        const float ref = m == -INFINITY ? 0.f : m * c2;
        const float fade = ex2(fmaf(top[i], c2, -ref));        // 0 while top is -infinity
        top[i] = m;
        float part = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[n][2 * i + e] = ex2(fmaf(s[n][2 * i + e], c2, -ref));
                part += s[n][2 * i + e];
            }
        sum[i] = fmaf(sum[i], fade, part);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            o[d][2 * i] *= fade;
            o[d][2 * i + 1] *= fade;
        }
    }
}

// ----------------------------------------------------------------------------- short sequences
//
// A block of four warps takes 64 rows in all: one tile of M = 64 rows of one head, or two or four heads of
// a tile of 32 or 16 rows, so that short sequences fill the warps.  Each warp owns 16 query rows.  Keys
// come in tiles of M.
constexpr int kShortThreads = 128;
template <int DP>
constexpr size_t short_smem() {
    return size_t(3) * 64 * DP * 2;
}

// Rows [0, M) of a tile (zeros past n and past D) by the threads of one unit.
template <class T, int DP, int M>
__device__ __forceinline__ void copy_tile(uint32_t dst, const void* src, long long stride, long long row0, int n, int D,
                                          int head, int tid, int threads) {
    for (int i = tid; i < M * (DP / 8); i += threads) {
        const int r = i / (DP / 8), c = i % (DP / 8);
        const bool take = r < n && c * 8 < D;
        const T* g = static_cast<const T*>(src) + (take ? (row0 + r) * stride + static_cast<long long>(head) * D + c * 8 : 0);
        cp_async16(at<DP>(dst, r, c), g, take);
    }
}

template <class T, int DP, int M>
__global__ void __launch_bounds__(kShortThreads) eqlin_attn_fwd_short_kernel(const Params p) {
    constexpr int U = 64 / M, WU = 4 / U, NT = M / 8;      // heads of a block, warps of a head
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_hb = (p.heads + U - 1) / U;
    const int unit = warp / WU, rw = warp % WU;
    const int h = (blockIdx.x % n_hb) * U + unit;
    const Tile t = find_tile<M>(p.q_offsets, p.sequences, p.q_rows, blockIdx.x / n_hb);
    if (t.tile < 0) return;
    const Rows kr = p.k_offsets == p.q_offsets && p.k_rows == p.q_rows ? t.own : sequence_rows(p.k_offsets, t.b, p.k_rows);
    const int r0 = t.tile * M, n = min(M, t.own.len - r0);
    const int seen = keys_seen(r0 + n - 1, t.own.len, kr.len, p.causal);
    const bool on = h < p.heads;                            // the last block may have fewer heads
    const int hk = h / (p.heads / p.kv_heads);
    const uint32_t sq = ptx::smem_u32(smem) + unit * (3 * M * DP * 2), sk = sq + M * DP * 2, sv = sk + M * DP * 2;
    const int tid = threadIdx.x - unit * WU * 32, nth = WU * 32;
    const int steps = (p.D + 15) / 16;
    const float c2 = p.scale * kLog2e;
    float o[DP / 8][4];
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    const int row = rw * 16 + (lane >> 2);                  // of the tile; and row + 8
    if (on) copy_tile<T, DP, M>(sq, p.q, p.q_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h, tid, nth);
    cp_async_commit();
    for (int k0 = 0; k0 < seen; k0 += M) {
        const int kn = min(M, kr.len - k0);
        if (k0 > 0) __syncthreads();
        if (on) {
            copy_tile<T, DP, M>(sk, p.k, p.k_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk, tid, nth);
            cp_async_commit();
            copy_tile<T, DP, M>(sv, p.v, p.v_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk, tid, nth);
            cp_async_commit();
        }
        cp_async_wait<1>();
        __syncthreads();
        float s[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
        const bool work = on && rw * 16 < n;
        if (work) {
            rows_by_rows<T, DP, NT>(s, sq + rw * 16 * (DP * 2), sk, steps, lane);
            int last[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int lim = p.causal ? r0 + row + 8 * i + 1 + kr.len - t.own.len - k0 : kn;
                last[i] = min(lim, kn);
            }
            softmax_step<NT, DP / 8>(s, o, top, sum, last, c2, lane);
        }
        cp_async_wait<0>();
        __syncthreads();
        if (work) weights_by_rows<T, DP, NT>(o, s, sv, p.D, lane);
    }
    cp_async_wait<0>();
    __syncthreads();
    if (!on) return;
    // outputs through shared memory (this warp's rows of Q), then as whole 16-byte chunks
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float l = quad_sum(sum[i]);
        const float inv = l == 0.f ? 0.f : 1.f / l;         // a row that sees no key
        const int r = row + 8 * i;
        if (p.lse && (lane & 3) == 0 && r < n)
            p.lse[static_cast<long long>(h) * p.q_rows + t.own.start + r0 + r] =
                l == 0.f ? -INFINITY : fmaf(top[i], p.scale, logf(l));
#pragma unroll
        for (int d = 0; d < DP / 8; ++d) {
            const uint32_t w = Io16<T>::pack(o[d][2 * i] * inv, o[d][2 * i + 1] * inv);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at<DP>(sq, r, d) + (lane & 3) * 4), "r"(w) : "memory");
        }
    }
    __syncwarp();
    const int chunks = p.D / 8;
    for (int i = lane; i < 16 * (DP / 8); i += 32) {
        const int r = rw * 16 + i / (DP / 8), c = i % (DP / 8);
        if (r >= n || c >= chunks) continue;
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(at<DP>(sq, r, c))
                     : "memory");
        *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (static_cast<long long>(t.own.start) + r0 + r) * p.o_stride +
                                  static_cast<long long>(h) * p.D + c * 8) = v;
    }
}

// ------------------------------------------------------------------- few queries over many keys
//
// The rows of a tile are the queries of one sequence for all query heads of one key head, query-major:
// packed row i * group + g.  A block takes 16 of them and one of `splits` slices of the keys; its warps
// take turns at blocks of 16 keys, each with its own ring of copies, and no barrier until their sums are
// joined in shared memory.  With several slices the block writes o and lse in fp32 to the workspace
// ([split][head][row]) and eqlin_attn_join_kernel joins them.
template <int DP>
struct Few {
    static constexpr int WARPS = 8;
    static constexpr int STAGES = DP == 64 ? 4 : 3;
    static constexpr int STAGE_BYTES = 2 * 16 * DP * 2;     // 16 keys of K, 16 of V
    static constexpr int Q_BYTES = 16 * DP * 2;
    static constexpr size_t RING = size_t(WARPS) * STAGES * STAGE_BYTES;
    static constexpr size_t JOIN = size_t(WARPS) * 16 * (DP + 4) * 4 + WARPS * 16 * 8;
    static constexpr size_t SMEM = Q_BYTES + (RING > JOIN ? RING : JOIN);
};

template <class T, int DP>
__global__ void __launch_bounds__(Few<DP>::WARPS * 32)
    eqlin_attn_fwd_few_kernel(const Params p) {
    using F = Few<DP>;
    const int splits = p.splits;
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.heads / p.kv_heads;
    const int split = blockIdx.x % splits, rest = blockIdx.x / splits;
    const int hk = rest % p.kv_heads;
    const Tile t = find_tile<16>(p.q_offsets, p.sequences, p.q_rows, rest / p.kv_heads, group);
    if (t.tile < 0) return;
    const Rows kr = sequence_rows(p.k_offsets, t.b, p.k_rows);
    const int r0 = t.tile * 16;                             // packed row
    const int n = min(16, t.own.len * group - r0);
    const int seen = keys_seen((r0 + n - 1) / group, t.own.len, kr.len, p.causal);
    // this slice's keys: blocks of 16, as evenly as possible
    const int blocks = (seen + 15) / 16;
    const int first = static_cast<int>(static_cast<long long>(blocks) * split / splits);
    const int end = static_cast<int>(static_cast<long long>(blocks) * (split + 1) / splits);
    const uint32_t sq = ptx::smem_u32(smem), ring = sq + F::Q_BYTES + warp * (F::STAGES * F::STAGE_BYTES);
    const int chunks = p.D / 8, steps = (p.D + 15) / 16;
    for (int i = threadIdx.x; i < 16 * (DP / 8); i += F::WARPS * 32) {
        const int r = i / (DP / 8), c = i % (DP / 8);
        const int q = (r0 + r) / group, h = hk * group + (r0 + r) - q * group;
        const bool take = r < n && c < chunks;
        cp_async16(at<DP>(sq, r, c),
                   static_cast<const T*>(p.q) + (take ? (static_cast<long long>(t.own.start) + q) * p.q_stride +
                                                            static_cast<long long>(h) * p.D + c * 8 : 0), take);
    }
    cp_async_commit();
    auto fetch = [&](int u) {                               // block u of this warp
        const int b = first + warp + u * F::WARPS;
        if (b < end) {
            const uint32_t dst = ring + (u % F::STAGES) * F::STAGE_BYTES;
            const int kn = kr.len - b * 16;
            copy_tile<T, DP, 16>(dst, p.k, p.k_stride, static_cast<long long>(kr.start) + b * 16, kn, p.D, hk, lane, 32);
            copy_tile<T, DP, 16>(dst + 16 * DP * 2, p.v, p.v_stride, static_cast<long long>(kr.start) + b * 16, kn, p.D, hk,
                                 lane, 32);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int u = 0; u < F::STAGES - 1; ++u) fetch(u);
    cp_async_wait<F::STAGES - 1>();
    __syncthreads();                                        // Q is there
    float o[DP / 8][4];
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    const float c2 = p.scale * kLog2e;
    const int row = lane >> 2;
    int lim[2];                                             // keys that each row sees
#pragma unroll
    for (int i = 0; i < 2; ++i) lim[i] = keys_seen((r0 + row + 8 * i) / group, t.own.len, kr.len, p.causal);
    for (int u = 0; first + warp + u * F::WARPS < end; ++u) {
        cp_async_wait<F::STAGES - 2>();
        __syncwarp();
        const int k0 = (first + warp + u * F::WARPS) * 16;
        const uint32_t kt = ring + (u % F::STAGES) * F::STAGE_BYTES;
        float s[2][4] = {};
        rows_by_rows<T, DP, 2>(s, sq, kt, steps, lane);
        const int last[2] = {min(lim[0], kr.len) - k0, min(lim[1], kr.len) - k0};
        softmax_step<2, DP / 8>(s, o, top, sum, last, c2, lane);
        weights_by_rows<T, DP, 2>(o, s, kt + 16 * DP * 2, p.D, lane);
        __syncwarp();
        fetch(u + F::STAGES - 1);
    }
    cp_async_wait<0>();
    __syncthreads();                                        // the rings are free
    // join the warps: o in fp32 [warp][16][DP + 4], maximum and sum [warp][16]
    float* jo = reinterpret_cast<float*>(smem + F::Q_BYTES);
    float2* jm = reinterpret_cast<float2*>(jo + F::WARPS * 16 * (DP + 4));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float l = quad_sum(sum[i]);
        if ((lane & 3) == 0) jm[warp * 16 + row + 8 * i] = make_float2(top[i], l);
#pragma unroll
        for (int d = 0; d < DP / 8; ++d)
            *reinterpret_cast<float2*>(jo + (warp * 16 + row + 8 * i) * (DP + 4) + d * 8 + (lane & 3) * 2) =
                make_float2(o[d][2 * i], o[d][2 * i + 1]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * (DP / 4); i += F::WARPS * 32) {
        const int r = i / (DP / 4), c = i % (DP / 4) * 4;
        if (r >= n || c >= p.D) continue;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < F::WARPS; ++w) m = fmaxf(m, jm[w * 16 + r].x);
        const float ref = m == -INFINITY ? 0.f : m * c2;
        float l = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < F::WARPS; ++w) {
            const float2 ms = jm[w * 16 + r];
            const float f = ex2(fmaf(ms.x, c2, -ref));
            const float4 b = *reinterpret_cast<const float4*>(jo + (w * 16 + r) * (DP + 4) + c);
            l = fmaf(f, ms.y, l);
            a.x = fmaf(f, b.x, a.x);
            a.y = fmaf(f, b.y, a.y);
            a.z = fmaf(f, b.z, a.z);
            a.w = fmaf(f, b.w, a.w);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int q = (r0 + r) / group, h = hk * group + (r0 + r) - q * group;
        const long long token = static_cast<long long>(t.own.start) + q;
        const float lse = l == 0.f ? -INFINITY : fmaf(m, p.scale, logf(l));
        const float v[4] = {a.x * inv, a.y * inv, a.z * inv, a.w * inv};
        if (splits == 1) {
            if (p.lse && c == 0) p.lse[static_cast<long long>(h) * p.q_rows + token] = lse;
            Vec<T, 4>::store(static_cast<T*>(p.out) + token * p.o_stride + static_cast<long long>(h) * p.D + c, Vec<T, 4>::pack(v));
        } else {
            const long long pr = (static_cast<long long>(split) * p.heads + h) * p.q_rows + token;
            if (c == 0) p.part_lse[pr] = lse;
            *reinterpret_cast<float4*>(p.part_o + pr * p.D + c) = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
}

}  // namespace mma

// o = sum_s exp(lse_s - lse) o_s,  lse = log sum_s exp(lse_s), over the slices of the keys: a group of 32
// threads for each row and head.  Rows that no sequence covers are left alone.
template <class T>
__global__ void __launch_bounds__(128) eqlin_attn_join_kernel(const Params p) {
    const int splits = p.splits;
    const float *part_o = p.part_o, *part_lse = p.part_lse;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (unit >= static_cast<long long>(p.q_rows) * p.heads) return;
    const int row = static_cast<int>(unit / p.heads), h = static_cast<int>(unit - static_cast<long long>(row) * p.heads);
    if (p.q_offsets && (row < p.q_offsets[0] || row >= p.q_offsets[p.sequences])) return;
    const long long pr = static_cast<long long>(h) * p.q_rows + row, step = static_cast<long long>(p.heads) * p.q_rows;
    float m = -INFINITY, nan = 0.f;
    for (int s = lane; s < splits; s += 32) {
        const float l = part_lse[pr + s * step];
        m = fmaxf(m, l);
        if (l != l) nan = l;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        nan += __shfl_xor_sync(0xFFFFFFFFu, nan, o);
    }
    const float ref = m == -INFINITY ? 0.f : m;
    float l = nan;
    float a[4] = {nan, nan, nan, nan};
    for (int s = 0; s < splits; ++s) {
        const float f = expf(part_lse[pr + s * step] - ref);
        l += f;
        if (lane * 4 < p.D && f > 0.f) {
            const float4 b = *reinterpret_cast<const float4*>(part_o + (pr + s * step) * p.D + lane * 4);
            a[0] = fmaf(f, b.x, a[0]);
            a[1] = fmaf(f, b.y, a[1]);
            a[2] = fmaf(f, b.z, a[2]);
            a[3] = fmaf(f, b.w, a[3]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (p.lse && lane == 0) p.lse[pr] = l == 0.f ? -INFINITY : m + logf(l);
    if (lane * 4 < p.D) {
        const float v[4] = {a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv};
        Vec<T, 4>::store(static_cast<T*>(p.out) + row * p.o_stride + static_cast<long long>(h) * p.D + lane * 4,
                         Vec<T, 4>::pack(v));
    }
}

}  // namespace attn
}  // namespace eqlin
