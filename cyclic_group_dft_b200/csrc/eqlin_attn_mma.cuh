// eqlin_attn_mma.cuh -- attention by 16-row warp products (mma.sync), whose scores and outputs stay in
// registers:
//   16-bit I/O where a 128-row tcgen05 tile would be mostly empty: short sequences (windows of a few dozen tokens)
//   and few queries over many keys.  Both are bound by memory, not by the tensor cores.
//   fp32 I/O of more than a few tiles, each product as three of tf32: with hi = tf32(v) (rounded to nearest) and
//   lo = v - hi (exact, at most 2^-11 |v|), a b = hi hi + hi lo + lo hi but for lo lo and what the tensor core
//   cuts off lo: 2.5 * 2^-21 |a b| at most.  Bound by the tensor cores' tf32 rate, a third of it, and by the
//   splitting; against CUDA cores: 784 tokens, 8 sequences, 8 heads of 64 features forward 322 to 228 us,
//   gradients 1056 to 783; 4096 tokens, 4 heads of 128 1060 to 741 and 3530 to 2995.  (Each small product
//   behind the last on the same accumulator: 262 and 929, 916 and 4781.)
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
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// v = hi + lo, hi with the 11 significant bits of tf32
struct Split {
    uint32_t hi, lo;
    __device__ __forceinline__ explicit Split(uint32_t v) {
        asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(__uint_as_float(v)));
        lo = __float_as_uint(__uint_as_float(v) - __uint_as_float(hi));
    }
};
// The tensor cores cut the low bits of an accumulator at each product, always towards zero, which adds up: over 8192
// keys to 1.5e-5 of o.  So sums of kExact pieces of 8 start from zero and are then added in fp32: o is within 6e-7,
// where a plain fp32 computation has 1.6e-6 (pieces of 64: 1.0e-6, and with more registers 843 for 783 us of gradients).
constexpr int kExact = 4;
// d[i] += a b[i] in fp32 precision for N tiles of 8 columns: the small products first, and each of the three over
// all tiles before the next, so that no product waits for the one before it.
template <int N>
__device__ __forceinline__ void mma_f32(float (*d)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                        const uint32_t (&b)[N][2]) {
    uint32_t bh[N][2], bl[N][2];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const Split v(b[i][e]);
            bh[i][e] = v.hi;
            bl[i][e] = v.lo;
        }
#pragma unroll
    for (int i = 0; i < N; ++i) mma1688(d[i], al, bh[i][0], bh[i][1]);
#pragma unroll
    for (int i = 0; i < N; ++i) mma1688(d[i], ah, bl[i][0], bl[i][1]);
#pragma unroll
    for (int i = 0; i < N; ++i) mma1688(d[i], ah, bh[i][0], bh[i][1]);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// RB: bytes of a row of a tile
template <class T, int DP>
constexpr int kRowBytes = DP * static_cast<int>(sizeof(T));
template <int RB>
__device__ __forceinline__ uint32_t at(uint32_t tile, int row, int chunk) {
    return tile + row * RB + ((chunk ^ (row & 7)) << 4);
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

// What a lane adds to a tile's address to read pieces of 16 rows x 32 bytes with ldmatrix (16 features of 16 bits,
// or 8 of fp32, whose fragments have the same places).  Tiles are aligned to their row bytes, rows r and r + 8
// have the same chunk order, and the chunks of piece k differ from those of piece 0 in address bits from 5 on
// alone: (base + lane part) ^ (k << 5) is the whole address computation.
template <int RB>
struct Lane {
    uint32_t a;   // rows 0-15 of the lower 16 bytes, then of the upper (operand A; B through a transpose)
    uint32_t b;   // rows 0-7 lower, rows 0-7 upper, rows 8-15 lower, rows 8-15 upper (operand B)
    __device__ __forceinline__ explicit Lane(int lane)
        : a((lane & 15) * RB + (((lane >> 4) ^ (lane & 7)) << 4)),
          b(((lane & 7) + ((lane >> 4) << 3)) * RB + ((((lane >> 3) & 1) ^ (lane & 7)) << 4)) {}
};

// acc[n8 tile] (16 rows of A x NT * 8 rows of B) += A B^T over the features, A and B row tiles; `steps` pieces of
// 32 bytes.
template <class T, int DP, int NT>
__device__ __forceinline__ void rows_by_rows(float (&acc)[NT][4], uint32_t a_tile, uint32_t b_tile, int steps,
                                             const Lane<kRowBytes<T, DP>>& at) {
    constexpr int RB = kRowBytes<T, DP>;
    const uint32_t la = a_tile + at.a, lb = b_tile + at.b;
    if constexpr (sizeof(T) == 4) {
#pragma unroll 1
        for (int k0 = 0; k0 < steps; k0 += kExact) {
            float part[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.f;
#pragma unroll
            for (int ks = k0; ks < k0 + kExact; ++ks) {      // (past the head's features: zeros)
                uint32_t a[4], ah[4], al[4], b[NT][2];
                ldm4(a, la ^ (ks << 5));
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t r[4];
                    ldm4(r, (lb ^ (ks << 5)) + n * 8 * RB);
                    b[n][0] = r[0];
                    b[n][1] = r[1];
                    b[n + 1][0] = r[2];
                    b[n + 1][1] = r[3];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Split v(a[e]);
                    ah[e] = v.hi;
                    al[e] = v.lo;
                }
                mma_f32<NT>(part, ah, al, b);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][e] += part[n][e];
        }
    } else {
        // the next pieces are on their way while these are multiplied
        uint32_t a[2][4], b[2][NT / 2][4];
        auto fetch = [&](int ks) {
            ldm4(a[ks & 1], la ^ (ks << 5));
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) ldm4(b[ks & 1][n], (lb ^ (ks << 5)) + n * 16 * RB);
        };
        fetch(0);
#pragma unroll
        for (int ks = 0; ks < RB / 32; ++ks) {
            if (ks >= steps) break;
            if (ks + 1 < RB / 32) fetch(ks + 1);      // (past the head's features: zeros)
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                mma16816<T>(acc[2 * n], a[ks & 1], b[ks & 1][n][0], b[ks & 1][n][1]);
                mma16816<T>(acc[2 * n + 1], a[ks & 1], b[ks & 1][n][2], b[ks & 1][n][3]);
            }
        }
    }
}
// o[feature tile] += W B for 16-bit weights: w[i] holds rows lane / 4 and lane / 4 + 8 of columns 8 i + 2 (lane & 3)
// and the next.
template <class T, int DP, int NT>
__device__ __forceinline__ void packed_by_rows(float (&o)[DP / 8][4], const uint32_t (&w)[NT][2], uint32_t b_tile, int steps,
                                               const Lane<kRowBytes<T, DP>>& at) {
    constexpr int RB = kRowBytes<T, DP>, GROUP = 4;   // pieces of 16 features in flight
    const uint32_t lb = b_tile + at.a;
#pragma unroll
    for (int kb = 0; kb < NT / 2; ++kb) {
        const uint32_t a[4] = {w[2 * kb][0], w[2 * kb][1], w[2 * kb + 1][0], w[2 * kb + 1][1]};
#pragma unroll
        for (int d0 = 0; d0 < DP / 16; d0 += GROUP) {
            if (d0 >= steps) break;
            uint32_t b[GROUP][4];
#pragma unroll
            for (int d = 0; d < GROUP; ++d) ldm4t(b[d], (lb ^ ((d0 + d) << 5)) + kb * 16 * RB);
#pragma unroll
            for (int d = 0; d < GROUP; ++d) {
                mma16816<T>(o[2 * (d0 + d)], a, b[d][0], b[d][1]);
                mma16816<T>(o[2 * (d0 + d) + 1], a, b[d][2], b[d][3]);
            }
        }
    }
}
// o[feature tile] += W B: W = 16 rows x NT * 8 weights from accumulators (rounded to T where T has 16 bits), B a row
// tile.  fp32: the accumulator's columns 2 t and 2 t + 1 of 8 stand at k = t and t + 4, so rows 2 t and 2 t + 1 of B
// are read there.
template <class T, int DP, int NT>
__device__ __forceinline__ void weights_by_rows(float (&o)[DP / 8][4], const float (&w)[NT][4], uint32_t b_tile, int steps,
                                                const Lane<kRowBytes<T, DP>>& at, int lane) {
    constexpr int RB = kRowBytes<T, DP>;
    if constexpr (sizeof(T) == 4) {
        // feature 8 d + lane / 4 of row 8 kb + 2 (lane & 3), and of the next row
        const int t2 = (lane & 3) * 2, in = (lane >> 2) & 3, up = lane >> 4;
        const uint32_t row0 = b_tile + t2 * RB + ((up ^ t2) << 4) + in * 4;
        const uint32_t row1 = b_tile + (t2 + 1) * RB + ((up ^ (t2 + 1)) << 4) + in * 4;
        constexpr int GROUP = 4;                      // tiles of 8 features at once
#pragma unroll
        for (int d0 = 0; d0 < DP / 8; d0 += GROUP) {
            if (d0 >= steps) break;
            float part[GROUP][4];
#pragma unroll
            for (int kb = 0; kb < NT; ++kb) {
                if (kb % kExact == 0) {
#pragma unroll
                    for (int d = 0; d < GROUP; ++d) part[d][0] = part[d][1] = part[d][2] = part[d][3] = 0.f;
                }
                uint32_t ah[4], al[4], b[GROUP][2];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Split v(__float_as_uint(w[kb][e == 1 ? 2 : e == 2 ? 1 : e]));
                    ah[e] = v.hi;
                    al[e] = v.lo;
                }
#pragma unroll
                for (int d = 0; d < GROUP; ++d) {
                    const uint32_t at_d = (d0 + d) << 5;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(b[d][0]) : "r"((row0 ^ at_d) + kb * 8 * RB) : "memory");
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(b[d][1]) : "r"((row1 ^ at_d) + kb * 8 * RB) : "memory");
                }
                mma_f32<GROUP>(part, ah, al, b);
                if (kb % kExact == kExact - 1 || kb == NT - 1) {
#pragma unroll
                    for (int d = 0; d < GROUP; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[d0 + d][e] += part[d][e];
                }
            }
        }
    } else {
        uint32_t a[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            a[i][0] = Io16<T>::pack(w[i][0], w[i][1]);
            a[i][1] = Io16<T>::pack(w[i][2], w[i][3]);
        }
        packed_by_rows<T, DP, NT>(o, a, b_tile, steps, at);
    }
}

// Running softmax of 16 rows x NT * 8 keys: masks keys >= last[i] (relative to this tile) of row i of
// the pair, which are all >= `masked` (the same for the warp), turns s into weights, and past the `first` tile
// moves the maximum and scales o and sum.
template <int NT, int DT>
__device__ __forceinline__ void softmax_step(float (&s)[NT][4], float (&o)[DT][4], float (&top)[2], float (&sum)[2],
                                             const int (&last)[2], int masked, bool first, float c2, int lane) {
    if (masked < NT * 8) {
        const int col0 = (lane & 3) * 2;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n * 8 + 8 <= masked) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col0 + n * 8 + (e & 1) >= last[e >> 1]) s[n][e] = -INFINITY;
        }
    }
    float fade[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float m = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n) m = fmaxf(m, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
        m = fmaxf(top[i], quad_max(m));
        // Two rounded products, so that fade is exactly 1 while the maximum stays: what one fused operation would
        // leave of their rounding, always the same way, is a drift over many tiles.
        const float ref = m == -INFINITY ? 0.f : __fmul_rn(m, c2);
        fade[i] = ex2(__fsub_rn(__fmul_rn(top[i], c2), ref));  // 0 while top is -infinity
        top[i] = m;
        float part = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[n][2 * i + e] = ex2(fmaf(s[n][2 * i + e], c2, -ref));
                part += s[n][2 * i + e];
            }
        sum[i] = first ? part : fmaf(sum[i], fade[i], part);
    }
    if (!first) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] *= fade[e >> 1];
    }
}

// ----------------------------------------------------------------------------- short sequences
//
// A block of four warps takes 64 rows in all: one tile of M = 64 rows of one head, or two or four heads of
// a tile of 32 or 16 rows, so that short sequences fill the warps.  Each warp owns 16 query rows.  Keys
// come in tiles of M.  A block's copies, products and stores follow one another, and the three to five blocks of an SM
// overlap: bound by that latency more than by memory.  Windows of 49 tokens, 4096 of them, 3 heads of 128 features:
// forward 143 us (4.3 TB/s; instructions issued in 51 % of the cycles), gradients 326 us (3.8 TB/s counting each
// tensor once), against 1450 us of a kernel for all lengths on the CUDA cores.  Several windows to a block, one after
// the other, gained nothing (143 to 147 us for 2 to 3).
constexpr int kShortThreads = 128;

// Most of these sequences have one tile, so the first tiles need no search: block b of the first `sequences` takes
// tile 0 of sequence b.  The later tiles of longer sequences have slots by their rows: tile t of sequence b is
// slot off[b] / M + t, one of rows / M that overlap nothing, and the blocks after the first ones look through
// kLaterSlots of them each.
constexpr int kLaterSlots = 8;
template <int M>
__host__ __device__ constexpr long long short_blocks(long long rows, long long sequences, long long per = 1) {
    return (sequences + per - 1) / per + (rows / M + kLaterSlots - 1) / kLaterSlots;
}
template <int M, class F>
__device__ __forceinline__ void later_tiles(const int32_t* offsets, int sequences, int rows, int block, F&& f) {
    const int first = block * kLaterSlots + 1;
    for (int slot = first; slot < first + kLaterSlots && slot <= rows / M; ++slot) {
        const Tile t = find_tile<M, true>(offsets, sequences, rows, slot);
        if (t.tile < 0) continue;
        f(t);
        __syncthreads();   // the next tile takes the same shared memory
    }
}
template <int M, class F>
__device__ __forceinline__ void for_short_tiles(const int32_t* offsets, int sequences, int rows, int block, F&& f) {
    if (block < sequences) {
        Tile t;
        t.b = block;
        t.own = sequence_rows(offsets, block, rows);
        t.tile = 0;
        if (t.own.len > 0) f(t);
        return;
    }
    later_tiles<M>(offsets, sequences, rows, block - sequences, f);
}
template <class T, int DP>
constexpr size_t short_smem() {
    return size_t(3) * 64 * kRowBytes<T, DP>;
}

// Rows [0, M) of a tile (zeros past n and past D) by THREADS threads: a thread keeps its 16-byte column.
template <class T, int DP, int M, int THREADS>
__device__ __forceinline__ void copy_tile(uint32_t dst, const void* src, long long stride, long long row0, int n, int D,
                                          int head, int tid) {
    constexpr int RB = kRowBytes<T, DP>, CHUNKS = RB / 16, PER = 16 / sizeof(T);
    constexpr int ROWS = THREADS / CHUNKS;                  // rows of one step
    const int c = tid % CHUNKS, r0 = tid / CHUNKS;
    const T* g = static_cast<const T*>(src) + (row0 + r0) * stride + static_cast<long long>(head) * D + c * PER;
    const long long step = ROWS * stride;
    const int left = c * PER < D ? n - r0 : 0;              // rows k * ROWS below this are copied
    const uint32_t d0 = at<RB>(dst, r0, c);
#pragma unroll
    for (int k = 0; k < M / ROWS; ++k) {
        const bool take = k * ROWS < left;
        const uint32_t d = ROWS % 8 == 0 ? d0 + k * ROWS * RB : at<RB>(dst, r0 + k * ROWS, c);
        cp_async16(d, take ? g : static_cast<const T*>(src), take);
        g += step;
    }
}

// Output rows of a warp, 16 bits through its 16 rows of a tile in shared memory and then as whole 16-byte chunks: the
// accumulators times mul[i] (row lane / 4 + 8 i), rows below n.
template <class T, int DP>
__device__ __forceinline__ void store_rows(const float (&acc)[DP / 8][4], const float (&mul)[2], uint32_t tile, int warp_row,
                                           int n, int D, T* out, long long stride, int lane) {
    if constexpr (sizeof(T) == 4) {   // four lanes write 32 bytes of a row: whole sectors as it is
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = warp_row + (lane >> 2) + 8 * i;
            if (r >= n) continue;
            float* row = out + r * stride + (lane & 3) * 2;
#pragma unroll
            for (int d = 0; d < DP / 8; ++d)
                if (d * 8 < D) *reinterpret_cast<float2*>(row + d * 8) = make_float2(acc[d][2 * i] * mul[i], acc[d][2 * i + 1] * mul[i]);
        }
    } else {
        constexpr int RB = kRowBytes<T, DP>;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t base = at<RB>(tile, warp_row + (lane >> 2) + 8 * i, 0) + (lane & 3) * 4;
#pragma unroll
            for (int d = 0; d < DP / 8; ++d) {
                const uint32_t w = Io16<T>::pack(acc[d][2 * i] * mul[i], acc[d][2 * i + 1] * mul[i]);
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(base ^ (d << 4)), "r"(w) : "memory");
            }
        }
        __syncwarp();
        constexpr int ROWS = 32 / (DP / 8);                     // rows of one step
        const int c = lane % (DP / 8);
#pragma unroll
        for (int k = 0; k < 16 / ROWS; ++k) {
            const int r = warp_row + lane / (DP / 8) + k * ROWS;
            if (r >= n || c * 8 >= D) continue;
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(at<RB>(tile, r, c))
                         : "memory");
            *reinterpret_cast<uint4*>(out + r * stride + c * 8) = v;
        }
    }
}

template <class T, int DP, int M>
__device__ __forceinline__ void fwd_short_tile(const Params& p, uint8_t* smem, int head_block, const Tile& t) {
    constexpr int RB = kRowBytes<T, DP>, U = 64 / M, WU = 4 / U, NT = M / 8;      // heads of a block, warps of a head
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = warp / WU, rw = warp % WU;
    const int h = (head_block) * U + unit;
    const Rows kr = other_rows(p, t, p.k_offsets, p.k_rows);
    const int r0 = t.tile * M, n = min(M, t.own.len - r0);
    const int seen = keys_seen(r0 + n - 1, t.own.len, kr.len, p.causal);
    const bool on = h < p.heads;                            // the last block may have fewer heads
    const int hk = h / (p.heads / p.kv_heads);
    const uint32_t sq = ptx::smem_u32(smem) + unit * (3 * M * RB), sk = sq + M * RB, sv = sk + M * RB;
    const int tid = threadIdx.x - unit * WU * 32;
    const Lane<RB> la(lane);
    const int steps = (p.D * static_cast<int>(sizeof(T)) + 31) / 32;
    const float c2 = p.scale * kLog2e;
    float o[DP / 8][4];
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    const int row = rw * 16 + (lane >> 2);                  // of the tile; and row + 8
    if (on) copy_tile<T, DP, M, WU * 32>(sq, p.q, p.q_stride, static_cast<long long>(t.own.start) + r0, n, p.D, h, tid);
    cp_async_commit();
    for (int k0 = 0; k0 < seen; k0 += M) {
        const int kn = min(M, kr.len - k0);
        if (k0 > 0) __syncthreads();
        if (on) {
            copy_tile<T, DP, M, WU * 32>(sk, p.k, p.k_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk, tid);
            cp_async_commit();
            copy_tile<T, DP, M, WU * 32>(sv, p.v, p.v_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk, tid);
            cp_async_commit();
        }
        cp_async_wait<1>();
        __syncthreads();
        float s[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
        const bool work = on && rw * 16 < n;
        if (work) {
            rows_by_rows<T, DP, NT>(s, sq + rw * 16 * RB, sk, steps, la);
            int last[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int lim = p.causal ? r0 + row + 8 * i + 1 - t.own.len + kr.len - k0 : kn;
                last[i] = min(lim, kn);
            }
            softmax_step<NT, DP / 8>(s, o, top, sum, last, p.causal ? 0 : kn, k0 == 0, c2, lane);
        }
        cp_async_wait<0>();
        __syncthreads();
        if (work) weights_by_rows<T, DP, NT>(o, s, sv, steps, la, lane);
    }
    cp_async_wait<0>();
    __syncthreads();
    if (!on) return;
    float inv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float l = quad_sum(sum[i]);
        inv[i] = l == 0.f ? 0.f : 1.f / l;                  // a row that sees no key
        if (p.lse && (lane & 3) == 0 && row + 8 * i < n)
            p.lse[static_cast<long long>(h) * p.q_rows + t.own.start + r0 + row + 8 * i] =
                l == 0.f ? -INFINITY : fmaf(top[i], p.scale, logf(l));
    }
    store_rows<T, DP>(o, inv, sq, rw * 16, n, p.D,
                      static_cast<T*>(p.out) + (static_cast<long long>(t.own.start) + r0) * p.o_stride +
                          static_cast<long long>(h) * p.D, p.o_stride, lane);
}
template <class T, int DP, int M>
__global__ void __launch_bounds__(kShortThreads, DP == 128 ? 4 : 5) eqlin_attn_fwd_short_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    constexpr int U = 64 / M;
    const int n_hb = (p.heads + U - 1) / U;
    for_short_tiles<M>(p.q_offsets, p.sequences, p.q_rows, blockIdx.x / n_hb,
                       [&](const Tile& t) { fwd_short_tile<T, DP, M>(p, smem, blockIdx.x % n_hb, t); });
}

// Gradients of short sequences: the forward's tiles, with four of them (Q, dO, K, V) in shared memory.
template <class T, int DP>
constexpr size_t short_bwd_smem() {
    return size_t(4) * 64 * kRowBytes<T, DP> + 2 * 64 * sizeof(float);
}

// fp16 (kLifted): ds of two rows, lifted so that the rows' largest values use the type's range.  The rows keep the
// exponents `lift`; where a tile has values of 2^15 and more with them, the sums `acc` (zeros while `fresh`) move to a
// smaller one, with two bits left so that this is rare.  Every lane of the warp must call it.
template <int NT, int DT>
__device__ __forceinline__ void lift_rows(float (&ds)[NT][4], float (&acc)[DT][4], int (&lift)[2], bool fresh) {
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) m[i] = fmaxf(m[i], fmaxf(fabsf(ds[n][2 * i]), fabsf(ds[n][2 * i + 1])));
    if (fresh || __any_sync(0xFFFFFFFFu, m[0] >= power_of_two(15 - lift[0]) || m[1] >= power_of_two(15 - lift[1]))) {
        float fade[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = min(lift[i], lift_of(quad_max(m[i])));
            fade[i] = power_of_two(e - lift[i]);
            lift[i] = e;
        }
        if (!fresh) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[d][e] *= fade[e >> 1];
        }
    }
    const float up[2] = {power_of_two(lift[0]), power_of_two(lift[1])};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) ds[n][e] *= up[e >> 1];
}

// Of the warp's 16 rows from `warp_row` on: off = -lse log2(e) and delta = do . o of rows lane / 4 and lane / 4 + 8.
template <class T, int RB>
__device__ __forceinline__ void row_stats(const Params& p, int h, long long first_row, int warp_row, int n, int lane,
                                          float (&off)[2], float (&delta)[2]) {
    // delta: two lanes a row, each half of its features
    const int r = warp_row + (lane >> 1);
    float sum = 0.f;
    if (r < n) {
        const T* po = static_cast<const T*>(p.o) + (first_row + r) * p.o_stride + static_cast<long long>(h) * p.D;
        const T* pd = static_cast<const T*>(p.dout) + (first_row + r) * p.do_stride + static_cast<long long>(h) * p.D;
#pragma unroll
        for (int c = 0; c < RB / 32; ++c) {
            constexpr int PER = 16 / sizeof(T);
            const int first = (2 * c + (lane & 1)) * PER;
            if (first >= p.D) break;
            float a[PER], b[PER];
            Vec<T, PER>::unpack(Vec<T, PER>::load(po + first), a);
            Vec<T, PER>::unpack(Vec<T, PER>::load(pd + first), b);
#pragma unroll
            for (int e = 0; e < PER; ++e) sum = fmaf(a[e], b[e], sum);
        }
    }
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
    const long long stat = static_cast<long long>(h) * p.q_rows + first_row;
    if (r < n && !(lane & 1)) p.delta[stat + r] = sum;
    const int row = warp_row + (lane >> 2);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        delta[i] = __shfl_sync(0xFFFFFFFFu, sum, (lane >> 2) * 2 + 16 * i);
        off[i] = 0.f;
        if (row + 8 * i < n) {
            const float l = p.lse[stat + row + 8 * i];
            off[i] = l == -INFINITY ? 0.f : -l * kLog2e;        // a row that sees no key: all of it is masked
        }
    }
}

// dq, and delta = do . o of its rows, which the kernel for dk and dv (launched next) reads.
template <class T, int DP, int M>
__device__ __forceinline__ void dq_short_tile(const Params& p, uint8_t* smem, int head_block, const Tile& t) {
    constexpr int RB = kRowBytes<T, DP>, U = 64 / M, WU = 4 / U, NT = M / 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = warp / WU, rw = warp % WU;
    const int h = (head_block) * U + unit;
    const Rows kr = other_rows(p, t, p.k_offsets, p.k_rows);
    const int r0 = t.tile * M, n = min(M, t.own.len - r0);
    const int seen = keys_seen(r0 + n - 1, t.own.len, kr.len, p.causal);
    const bool on = h < p.heads;
    const int hk = h / (p.heads / p.kv_heads);
    const uint32_t sq = ptx::smem_u32(smem) + unit * (4 * M * RB), sdo = sq + M * RB, sk = sdo + M * RB,
                   sv = sk + M * RB;
    const int tid = threadIdx.x - unit * WU * 32;
    const Lane<RB> la(lane);
    const int steps = (p.D * static_cast<int>(sizeof(T)) + 31) / 32;
    const float c2 = p.scale * kLog2e;
    const int row = rw * 16 + (lane >> 2);
    const long long first_row = static_cast<long long>(t.own.start) + r0;
    float dq[DP / 8][4];
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) dq[d][0] = dq[d][1] = dq[d][2] = dq[d][3] = 0.f;
    float off[2] = {0.f, 0.f}, delta[2];
    int lift[2] = {kLiftMost, kLiftMost};
    if (on) {
        copy_tile<T, DP, M, WU * 32>(sq, p.q, p.q_stride, first_row, n, p.D, h, tid);
        copy_tile<T, DP, M, WU * 32>(sdo, p.dout, p.do_stride, first_row, n, p.D, h, tid);
        row_stats<T, RB>(p, h, first_row, rw * 16, n, lane, off, delta);
    }
    for (int k0 = 0; k0 < seen; k0 += M) {
        const int kn = min(M, kr.len - k0);
        if (k0 > 0) __syncthreads();
        if (on) {
            copy_tile<T, DP, M, WU * 32>(sk, p.k, p.k_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk, tid);
            copy_tile<T, DP, M, WU * 32>(sv, p.v, p.v_stride, static_cast<long long>(kr.start) + k0, kn, p.D, hk, tid);
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        if (!on || rw * 16 >= n) continue;
        float s[NT][4], dp[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] = dp[i][e] = 0.f;
        rows_by_rows<T, DP, NT>(s, sq + rw * 16 * RB, sk, steps, la);
        rows_by_rows<T, DP, NT>(dp, sdo + rw * 16 * RB, sv, steps, la);
        int last[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) last[i] = min(kn, p.causal ? r0 + row + 8 * i + 1 - t.own.len + kr.len - k0 : kn);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool vis = i * 8 + (lane & 3) * 2 + (e & 1) < last[e >> 1];
                s[i][e] = vis ? ex2(fmaf(s[i][e], c2, off[e >> 1])) * (dp[i][e] - delta[e >> 1]) : 0.f;
            }
        if constexpr (kLifted<T>) lift_rows<NT, DP / 8>(s, dq, lift, k0 == 0);
        weights_by_rows<T, DP, NT>(dq, s, sk, steps, la, lane);
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    if (!on) return;
    float mul[2] = {p.scale, p.scale};
    if constexpr (kLifted<T>) {
#pragma unroll
        for (int i = 0; i < 2; ++i) mul[i] *= power_of_two(-lift[i]);
    }
    store_rows<T, DP>(dq, mul, sq, rw * 16, n, p.D,
                      static_cast<T*>(p.dq) + first_row * p.dq_stride + static_cast<long long>(h) * p.D, p.dq_stride, lane);
}
// o[feature tile] += W^T B over the n rows of W (16-bit weights, one row of RB bytes each, columns rw * 16 on) and of
// B (a row tile).
template <class T, int DP, int M>
__device__ __forceinline__ void columns_by_rows(float (&o)[DP / 8][4], uint32_t w_tile, int rw, uint32_t b_tile, int n,
                                                int steps, const Lane<kRowBytes<T, DP>>& at) {
    constexpr int RB = kRowBytes<T, DP>, GROUP = 4;
    const uint32_t lw = (w_tile + at.b) ^ (rw << 5), lb = b_tile + at.a;
#pragma unroll
    for (int kb = 0; kb < M / 16; ++kb) {
        if (kb * 16 >= n) break;
        uint32_t a[4];
        ldm4t(a, lw + kb * 16 * RB);
#pragma unroll
        for (int d0 = 0; d0 < DP / 16; d0 += GROUP) {
            if (d0 >= steps) break;
            uint32_t b[GROUP][4];
#pragma unroll
            for (int d = 0; d < GROUP; ++d) ldm4t(b[d], (lb ^ ((d0 + d) << 5)) + kb * 16 * RB);
#pragma unroll
            for (int d = 0; d < GROUP; ++d) {
                mma16816<T>(o[2 * (d0 + d)], a, b[d][0], b[d][1]);
                mma16816<T>(o[2 * (d0 + d) + 1], a, b[d][2], b[d][3]);
            }
        }
    }
}

// Whether a sequence's gradients are all computed from one tile: one head of keys for each of queries, and no more
// than M rows on either side.
template <int M>
__device__ __forceinline__ bool one_tile(const Params& p, int queries, int keys) {
    return p.heads == p.kv_heads && queries > 0 && queries <= M && keys > 0 && keys <= M;
}

// All gradients of one head of a sequence of one tile: the scores and the weights are computed once, by warps that
// own 16 queries; the weights and ds go to shared memory (over V and K, which are then done with), for warps
// that own 16 keys.  Five products and each tensor read once, for seven and twice with dq and dk, dv apart (windows
// of 49, 3 heads of 128: 326 us for 587).  Q and K are waited for first; dO, V and the rows of O for delta arrive
// while the scores are computed (all at once: 485 us).
template <class T, int DP, int M>
__device__ __forceinline__ void bwd_one_tile(const Params& p, uint8_t* smem, int head_block, const Tile& t, const Rows& kr) {
    constexpr int RB = kRowBytes<T, DP>, U = 64 / M, WU = 4 / U, NT = M / 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = warp / WU, rw = warp % WU;
    const int h = head_block * U + unit;
    const int n = t.own.len, kn = kr.len;
    const bool on = h < p.heads, work = on && rw * 16 < n, key_work = on && rw * 16 < kn;
    const uint32_t sq = ptx::smem_u32(smem) + unit * (4 * M * RB), sdo = sq + M * RB, sk = sdo + M * RB,
                   sv = sk + M * RB;
    const int tid = threadIdx.x - unit * WU * 32;
    const Lane<RB> la(lane);
    const int steps = (p.D * static_cast<int>(sizeof(T)) + 31) / 32;
    const float c2 = p.scale * kLog2e;
    const int row = rw * 16 + (lane >> 2);
    const long long first_row = t.own.start, first_key = kr.start, col = static_cast<long long>(h) * p.D;
    // two lanes a row for delta: their half of the row of O is on its way while the scores are computed
    const int dr = rw * 16 + (lane >> 1);
    uint4 o[RB / 32];
    float off[2] = {0.f, 0.f};
    if (on) {
        copy_tile<T, DP, M, WU * 32>(sq, p.q, p.q_stride, first_row, n, p.D, h, tid);
        copy_tile<T, DP, M, WU * 32>(sk, p.k, p.k_stride, first_key, kn, p.D, h, tid);
    }
    cp_async_commit();
    if (on) {
        copy_tile<T, DP, M, WU * 32>(sdo, p.dout, p.do_stride, first_row, n, p.D, h, tid);
        copy_tile<T, DP, M, WU * 32>(sv, p.v, p.v_stride, first_key, kn, p.D, h, tid);
    }
    cp_async_commit();
    const T* po = static_cast<const T*>(p.o) + (first_row + dr) * p.o_stride + col;
#pragma unroll
    for (int c = 0; c < RB / 32; ++c) {
        const int first = (2 * c + (lane & 1)) * 8;
        o[c] = on && dr < n && first < p.D ? *reinterpret_cast<const uint4*>(po + first) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (on && row + 8 * i < n) {
            const float l = p.lse[static_cast<long long>(h) * p.q_rows + first_row + row + 8 * i];
            // a row that sees no key: all of it is masked
            off[i] = l == -INFINITY ? 0.f : fmaf(-l, kLog2e, kLiftOf<T>);
        }
    float s[NT][4], dp[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = dp[i][e] = 0.f;
    cp_async_wait<1>();
    __syncthreads();
    if (work) rows_by_rows<T, DP, NT>(s, sq + rw * 16 * RB, sk, steps, la);
    cp_async_wait<0>();
    __syncthreads();
    float dq[DP / 8][4], acc[DP / 8][4];
    uint32_t w[NT][2], ds[NT][2];
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) dq[d][0] = dq[d][1] = dq[d][2] = dq[d][3] = 0.f;
    int lift[2] = {kLiftMost, kLiftMost};                   // fp16: of the rows for dq, and one of the head for dk
    int* least = reinterpret_cast<int*>(smem + 4 * 64 * RB);      // the warps' smallest exponents
    if (work) {
        float sum = 0.f, delta[2];
#pragma unroll
        for (int c = 0; c < RB / 32; ++c) {
            uint4 d;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(d.x), "=r"(d.y), "=r"(d.z), "=r"(d.w)
                         : "r"(at<RB>(sdo, dr, 2 * c + (lane & 1)))
                         : "memory");
            float a[8], b[8];
            Vec<T, 8>::unpack(o[c], a);
            Vec<T, 8>::unpack(d, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(a[e], b[e], sum);
        }
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) delta[i] = __shfl_sync(0xFFFFFFFFu, sum, (lane >> 2) * 2 + 16 * i);
        rows_by_rows<T, DP, NT>(dp, sdo + rw * 16 * RB, sv, steps, la);
        int last[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) last[i] = min(kn, p.causal ? row + 8 * i + 1 + kn - n : kn);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool vis = i * 8 + (lane & 3) * 2 + (e & 1) < last[e >> 1];
                s[i][e] = vis ? ex2(fmaf(s[i][e], c2, off[e >> 1])) : 0.f;
                dp[i][e] = vis ? s[i][e] * (dp[i][e] - delta[e >> 1]) : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[i][e] = Io16<T>::pack(s[i][2 * e], s[i][2 * e + 1]);
                if constexpr (!kLifted<T>) ds[i][e] = Io16<T>::pack(dp[i][2 * e], dp[i][2 * e + 1]);
            }
        }
        if constexpr (kLifted<T>) {
            lift_rows<NT, DP / 8>(dp, dq, lift, true);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) ds[i][e] = Io16<T>::pack(dp[i][2 * e], dp[i][2 * e + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NT; ++i) w[i][0] = w[i][1] = ds[i][0] = ds[i][1] = 0;
    }
    if constexpr (kLifted<T>) {
        // (rows that do not exist or have ds = 0 keep the largest exponent)
        int e = work ? min(lift[0], lift[1]) : kLiftMost;
        e = __reduce_min_sync(0xFFFFFFFFu, e);
        if (lane == 0) least[warp] = e;
    }
    if (work) packed_by_rows<T, DP, NT>(dq, ds, sk, steps, la);
    __syncthreads();
    int lift_dk = 0;
    if constexpr (kLifted<T>) {
        lift_dk = kLiftMost;
#pragma unroll
        for (int i = 0; i < WU; ++i) lift_dk = min(lift_dk, least[unit * WU + i]);
        if (work) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // a second rounding only of what is subnormal then
                const __half2 f = __float2half2_rn(power_of_two(lift_dk - lift[e]));
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const __half2 d = __hmul2(reinterpret_cast<const __half2&>(ds[i][e]), f);
                    ds[i][e] = reinterpret_cast<const uint32_t&>(d);
                }
            }
        }
    }
    if (work) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t pw = at<RB>(sv, row + 8 * e, 0) + (lane & 3) * 4, pds = at<RB>(sk, row + 8 * e, 0) + (lane & 3) * 4;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(pw ^ (i << 4)), "r"(w[i][e]) : "memory");
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(pds ^ (i << 4)), "r"(ds[i][e]) : "memory");
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
    if (key_work) columns_by_rows<T, DP, M>(acc, sv, rw, sdo, n, steps, la);
    __syncthreads();
    float mul_dq[2] = {p.scale, p.scale}, mul[2] = {p.scale, p.scale}, one[2] = {1.f, 1.f};
    if constexpr (kLifted<T>) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {                       // ds holds the lift of p as well
            mul_dq[i] *= power_of_two(-lift[i] - kLiftP);
            mul[i] *= power_of_two(-lift_dk - kLiftP);
            one[i] = power_of_two(-kLiftP);
        }
    }
    // over the weights and dO, which all warps are done with; each warp in its own rows
    if (work) store_rows<T, DP>(dq, mul_dq, sv, rw * 16, n, p.D, static_cast<T*>(p.dq) + first_row * p.dq_stride + col, p.dq_stride, lane);
    if (key_work) {
        store_rows<T, DP>(acc, one, sdo, rw * 16, kn, p.D, static_cast<T*>(p.dv) + first_key * p.dv_stride + col, p.dv_stride, lane);
#pragma unroll
        for (int d = 0; d < DP / 8; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
        columns_by_rows<T, DP, M>(acc, sk, rw, sq, n, steps, la);
        __syncwarp();
        store_rows<T, DP>(acc, mul, sdo, rw * 16, kn, p.D, static_cast<T*>(p.dk) + first_key * p.dk_stride + col, p.dk_stride, lane);
    }
}
template <class T, int DP, int M>
__global__ void __launch_bounds__(kShortThreads, DP == 128 ? 3 : 4) eqlin_attn_dq_short_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    constexpr int U = 64 / M;
    const int n_hb = (p.heads + U - 1) / U;
    for_short_tiles<M>(p.q_offsets, p.sequences, p.q_rows, blockIdx.x / n_hb, [&](const Tile& t) {
        const Rows kr = other_rows(p, t, p.k_offsets, p.k_rows);
        if (one_tile<M>(p, t.own.len, kr.len)) bwd_one_tile<T, DP, M>(p, smem, blockIdx.x % n_hb, t, kr);
        else dq_short_tile<T, DP, M>(p, smem, blockIdx.x % n_hb, t);
    });
}

// dk and dv: a warp owns 16 keys; the query rows that see the tile pass by, for each head of the group.
template <class T, int DP, int M>
__device__ __forceinline__ void dkv_short_tile(const Params& p, uint8_t* smem, int head_block, const Tile& t) {
    constexpr int RB = kRowBytes<T, DP>, U = 64 / M, WU = 4 / U, NT = (M < 32 ? M : 32) / 8;   // queries in steps of 32 (or M) columns
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.heads / p.kv_heads;
    const int unit = warp / WU, rw = warp % WU;
    const int hk = (head_block) * U + unit;
    const Rows qr = other_rows(p, t, p.q_offsets, p.q_rows);
    const int r0 = t.tile * M, n = min(M, t.own.len - r0);
    const bool on = hk < p.kv_heads;
    const uint32_t sk = ptx::smem_u32(smem) + unit * (4 * M * RB), sv = sk + M * RB, sq = sv + M * RB,
                   sdo = sq + M * RB;
    float* slse = reinterpret_cast<float*>(smem + 4 * 64 * RB) + unit * 2 * M;   // lse, then delta, of the tile's rows
    float* sdelta = slse + M;
    const int tid = threadIdx.x - unit * WU * 32;
    const Lane<RB> la(lane);
    const int steps = (p.D * static_cast<int>(sizeof(T)) + 31) / 32;
    const float c2 = p.scale * kLog2e;
    const int key = r0 + rw * 16 + (lane >> 2);
    const long long first_row = static_cast<long long>(t.own.start) + r0;
    float dk[DP / 8][4], dv[DP / 8][4];
    int lift[2] = {kLiftMost, kLiftMost};
#pragma unroll
    for (int d = 0; d < DP / 8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) dk[d][e] = dv[d][e] = 0.f;
    if (on) {
        copy_tile<T, DP, M, WU * 32>(sk, p.k, p.k_stride, first_row, n, p.D, hk, tid);
        copy_tile<T, DP, M, WU * 32>(sv, p.v, p.v_stride, first_row, n, p.D, hk, tid);
    }
    const int begin = first_query(r0, qr.len, t.own.len, p.causal) / M * M;
    for (int g = 0; g < group; ++g) {
        const int h = hk * group + g;
        for (int q0 = begin; q0 < qr.len; q0 += M) {
            const int qn = min(M, qr.len - q0);
            if (g > 0 || q0 > begin) __syncthreads();
            if (on) {
                copy_tile<T, DP, M, WU * 32>(sq, p.q, p.q_stride, static_cast<long long>(qr.start) + q0, qn, p.D, h, tid);
                copy_tile<T, DP, M, WU * 32>(sdo, p.dout, p.do_stride, static_cast<long long>(qr.start) + q0, qn, p.D, h, tid);
                for (int i = tid; i < M; i += WU * 32) {
                    const long long stat = static_cast<long long>(h) * p.q_rows + qr.start + q0 + i;
                    const float l = i < qn ? p.lse[stat] : -INFINITY;
                    slse[i] = l == -INFINITY ? INFINITY : fmaf(l, kLog2e, -kLiftOf<T>);      // weights of zero
                    sdelta[i] = i < qn ? p.delta[stat] : 0.f;
                }
            }
            cp_async_commit();
            cp_async_wait<0>();
            __syncthreads();
            if (!on || rw * 16 >= n) continue;
#pragma unroll 1
            for (int c0 = 0; c0 < qn; c0 += NT * 8) {
                float s[NT][4], dp[NT][4];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][e] = dp[i][e] = 0.f;
                rows_by_rows<T, DP, NT>(s, sk + rw * 16 * RB, sq + c0 * RB, steps, la);
                rows_by_rows<T, DP, NT>(dp, sv + rw * 16 * RB, sdo + c0 * RB, steps, la);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int c = c0 + i * 8 + (lane & 3) * 2;
                    const float2 l = *reinterpret_cast<const float2*>(slse + c), dl = *reinterpret_cast<const float2*>(sdelta + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float w = ex2(fmaf(s[i][e], c2, e & 1 ? -l.y : -l.x));
                        // key j is seen by queries from j - (keys - queries) on
                        if (p.causal && q0 + c + (e & 1) < key + 8 * (e >> 1) - (t.own.len - qr.len)) w = 0.f;
                        s[i][e] = w;
                        dp[i][e] = w == 0.f ? 0.f : w * (dp[i][e] - (e & 1 ? dl.y : dl.x));
                    }
                }
                if constexpr (kLifted<T>) lift_rows<NT, DP / 8>(dp, dk, lift, g == 0 && q0 == begin && c0 == 0);
                weights_by_rows<T, DP, NT>(dv, s, sdo + c0 * RB, steps, la, lane);
                weights_by_rows<T, DP, NT>(dk, dp, sq + c0 * RB, steps, la, lane);
            }
        }
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    if (!on) return;
    float mul[2] = {p.scale, p.scale}, one[2] = {1.f, 1.f};
    if constexpr (kLifted<T>) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {                       // ds holds the lift of p as well
            mul[i] *= power_of_two(-lift[i] - kLiftP);
            one[i] = power_of_two(-kLiftP);
        }
    }
    const long long col = static_cast<long long>(hk) * p.D;
    store_rows<T, DP>(dk, mul, sk, rw * 16, n, p.D, static_cast<T*>(p.dk) + first_row * p.dk_stride + col, p.dk_stride, lane);
    store_rows<T, DP>(dv, one, sv, rw * 16, n, p.D, static_cast<T*>(p.dv) + first_row * p.dv_stride + col, p.dv_stride, lane);
}
// `per` (at most 32) sequences' first tiles to a block: most have been done by bwd_one_tile, and a block of this kernel
// that finds nothing to do costs as much as its launch (windows of 49, 4096 sequences, 3 heads of 128: 41 us in
// 13.5 thousand blocks).
template <class T, int DP, int M>
__global__ void __launch_bounds__(kShortThreads, DP == 128 ? 2 : 4) eqlin_attn_dkv_short_kernel(const Params p, int per) {
    extern __shared__ __align__(1024) uint8_t smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    constexpr int U = 64 / M;
    const int n_hb = (p.kv_heads + U - 1) / U, block = blockIdx.x / n_hb, hb = blockIdx.x % n_hb;
    const int first_blocks = (p.sequences + per - 1) / per;
    if (block < first_blocks) {
        const int lane = threadIdx.x & 31, b = block * per + lane;
        bool todo = lane < per && b < p.sequences;
        if (todo) {
            const Rows kr = sequence_rows(p.k_offsets, b, p.k_rows), qr = sequence_rows(p.q_offsets, b, p.q_rows);
            todo = kr.len > 0 && !one_tile<M>(p, qr.len, kr.len);
        }
        for (unsigned left = __ballot_sync(0xFFFFFFFFu, todo); left; left &= left - 1) {
            Tile t;
            t.b = block * per + __ffs(left) - 1;
            t.own = sequence_rows(p.k_offsets, t.b, p.k_rows);
            t.tile = 0;
            dkv_short_tile<T, DP, M>(p, smem, hb, t);
            __syncthreads();   // the next tile takes the same shared memory
        }
        return;
    }
    later_tiles<M>(p.k_offsets, p.sequences, p.k_rows, block - first_blocks,
                   [&](const Tile& t) { dkv_short_tile<T, DP, M>(p, smem, hb, t); });
}

// fp32 of every length: a block for each tile of 64 rows and head.  The kernels are bound by the three tf32
// products (503 multiply-adds a cycle and SM measured, so 168 of fp32; the FMA pipes have 124).
template <int DP>
__global__ void __launch_bounds__(kShortThreads) eqlin_attn_fwd_f32_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int slot = p.causal ? gridDim.x / p.heads - 1 - blockIdx.x / p.heads : blockIdx.x / p.heads;   // long rows first
    const Tile t = find_tile<64>(p.q_offsets, p.sequences, p.q_rows, slot);
    if (t.tile >= 0) fwd_short_tile<float, DP, 64>(p, smem, blockIdx.x % p.heads, t);
}
template <int DP>
__global__ void __launch_bounds__(kShortThreads) eqlin_attn_dq_f32_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int slot = p.causal ? gridDim.x / p.heads - 1 - blockIdx.x / p.heads : blockIdx.x / p.heads;
    const Tile t = find_tile<64>(p.q_offsets, p.sequences, p.q_rows, slot);
    if (t.tile >= 0) dq_short_tile<float, DP, 64>(p, smem, blockIdx.x % p.heads, t);
}
template <int DP>
__global__ void __launch_bounds__(kShortThreads) eqlin_attn_dkv_f32_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const Tile t = find_tile<64>(p.k_offsets, p.sequences, p.k_rows, blockIdx.x / p.kv_heads);
    if (t.tile >= 0) dkv_short_tile<float, DP, 64>(p, smem, blockIdx.x % p.kv_heads, t);
}

// ------------------------------------------------------------------- few queries over many keys
//
// The rows of a tile are the queries of one sequence for all query heads of one key head, query-major:
// packed row i * group + g.  A block takes 16 of them and one of `splits` slices of the keys; its warps
// take turns at blocks of KEYS keys, each with its own ring of copies, and no barrier until their sums are
// joined in shared memory.  With several slices the block writes o and lse in fp32 to the workspace
// ([split][head][row]) and eqlin_attn_join_kernel joins them.
//
// Bound by memory: each key and value is read once.  Per SM about 128 KB of copies are in flight.  One query, 8
// sequences of 16384 keys, 8 heads on 2 key heads of 64 features: 17 us with the join for 67 MB (3.9 TB/s; a launch,
// the offsets' reads and the join are 6 of them).
template <int DP>
struct Few {
    static constexpr int WARPS = 8;
    static constexpr int KEYS = DP == 64 ? 32 : 16;
    static constexpr int STAGES = 3;
    static constexpr int STAGE_BYTES = 2 * KEYS * DP * 2;   // K, then V
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
    extern __shared__ __align__(1024) uint8_t smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.heads / p.kv_heads;
    const int split = blockIdx.x % splits, rest = blockIdx.x / splits;
    const int hk = rest % p.kv_heads;
    const Tile t = find_tile<16>(p.q_offsets, p.sequences, p.q_rows, rest / p.kv_heads, group);
    if (t.tile < 0) return;
    const Rows kr = other_rows(p, t, p.k_offsets, p.k_rows);
    const int r0 = t.tile * 16;                             // packed row
    const int n = min(16, t.own.len * group - r0);
    const int seen = keys_seen((r0 + n - 1) / group, t.own.len, kr.len, p.causal);
    // this slice's keys: whole blocks, as evenly as possible
    const int blocks = (seen + F::KEYS - 1) / F::KEYS;
    const int first = static_cast<int>(static_cast<long long>(blocks) * split / splits);
    const int end = static_cast<int>(static_cast<long long>(blocks) * (split + 1) / splits);
    const uint32_t sq = ptx::smem_u32(smem), ring = sq + F::Q_BYTES + warp * (F::STAGES * F::STAGE_BYTES);
    const int chunks = p.D / 8, steps = (p.D + 15) / 16;
    const Lane<kRowBytes<T, DP>> la(lane);
    for (int i = threadIdx.x; i < 16 * (DP / 8); i += F::WARPS * 32) {
        const int r = i / (DP / 8), c = i % (DP / 8);
        const int q = (r0 + r) / group, h = hk * group + (r0 + r) - q * group;
        const bool take = r < n && c < chunks;
        cp_async16(at<kRowBytes<T, DP>>(sq, r, c),
                   static_cast<const T*>(p.q) + (take ? (static_cast<long long>(t.own.start) + q) * p.q_stride +
                                                            static_cast<long long>(h) * p.D + c * 8 : 0), take);
    }
    cp_async_commit();
    auto fetch = [&](int u) {                               // block u of this warp
        const int b = first + warp + u * F::WARPS;
        if (b < end) {
            const uint32_t dst = ring + (u % F::STAGES) * F::STAGE_BYTES;
            const int kn = kr.len - b * F::KEYS;
            const long long row0 = static_cast<long long>(kr.start) + static_cast<long long>(b) * F::KEYS;
            copy_tile<T, DP, F::KEYS, 32>(dst, p.k, p.k_stride, row0, kn, p.D, hk, lane);
            copy_tile<T, DP, F::KEYS, 32>(dst + F::STAGE_BYTES / 2, p.v, p.v_stride, row0, kn, p.D, hk, lane);
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
    const int seen_all = keys_seen(r0 / group, t.own.len, kr.len, p.causal);   // by every row
    for (int u = 0; first + warp + u * F::WARPS < end; ++u) {
        cp_async_wait<F::STAGES - 2>();
        __syncwarp();
        const int k0 = (first + warp + u * F::WARPS) * F::KEYS;
        const uint32_t kt = ring + (u % F::STAGES) * F::STAGE_BYTES;
        float s[F::KEYS / 8][4] = {};
        rows_by_rows<T, DP, F::KEYS / 8>(s, sq, kt, steps, la);
        const int last[2] = {min(lim[0], kr.len) - k0, min(lim[1], kr.len) - k0};
        softmax_step<F::KEYS / 8, DP / 8>(s, o, top, sum, last, min(seen_all - k0, F::KEYS), u == 0, c2, lane);
        weights_by_rows<T, DP, F::KEYS / 8>(o, s, kt + F::STAGE_BYTES / 2, steps, la, lane);
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
