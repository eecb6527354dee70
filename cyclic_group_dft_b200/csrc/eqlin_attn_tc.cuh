// eqlin_attn_tc.cuh -- 16-bit attention on the tcgen05 tensor cores: what the forward and the
// gradient kernels share, and the forward.
//
// Operands in shared memory are tiles of 128 token rows, one box of 64 features (128 bytes) after the
// other, as a TMA load with 128-byte swizzle leaves them.  The same tile serves a product over
// features (K-major: rows are the M or N index) and a product over tokens (MN-major: rows are the K
// index).  Features past the head's end arrive as zeros.
#pragma once

#include <cuda.h>

#include "eqlin_attn.cuh"

namespace eqlin {
namespace attn {

// Error word of this library's attention kernels on a device (bounded waits that ran out).
__device__ int g_status;

namespace tc {

constexpr int kTile = 128;                       // token rows of an operand tile
constexpr int kBoxBytes = kTile * 128;           // one box: 128 rows of 64 features
constexpr int kErrTimeout = -6;                  // EQLIN_ERR_TIMEOUT
constexpr int kErrMisaligned = -3;               // EQLIN_ERR_MISALIGNED
constexpr uint32_t kWaitSleepNs = 20000;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Ctl {
    volatile int abort;
    uint32_t tmem_base;
};

// Bounded mbarrier wait.  Returns false (after flagging) on timeout or abort.  The limit is counted in SM
// cycles, two for each nanosecond (the SM clock is below 2 GHz).
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, Ctl* ctl, unsigned long long timeout_ns) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t spin = 1;; ++spin) {
        if (ptx::mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) return true;
        if ((spin & 7u) == 0) {
            if (ctl->abort) return false;
            if (static_cast<unsigned long long>(clock64() - t0) > 2 * timeout_ns) {
                ctl->abort = 1;
                atomicCAS(&g_status, 0, kErrTimeout);
                return false;
            }
        }
    }
}
// The same for a whole warp: one answer for all lanes, which are together again afterwards.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, Ctl* ctl, unsigned long long timeout_ns) {
    return __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, ctl, timeout_ns));
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(is));
    return is != 0;
}
// One arrival for a whole warp (all lanes' work before it included): 32 single ones on one barrier would be
// carried out one after the other.
__device__ __forceinline__ void arrive_warp(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
}
// Bounded wait that ignores the abort flag, for copies or MMAs in flight before exit.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, unsigned long long timeout_ns) {
    if (ptx::mbar_try_wait(bar, parity)) return;
    const long long t0 = clock64();
    while (!ptx::mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) {
        if (static_cast<unsigned long long>(clock64() - t0) > 2 * timeout_ns) {
            atomicCAS(&g_status, 0, kErrTimeout);
            return;
        }
    }
}

// 3-D tiled TMA load of a box (feature, head, row).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int32_t c0, int32_t c1, int32_t c2,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], kind::f16; A: lane = row, two K elements per 32-bit column.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Descriptors of a tile, split in halves (the low half carries the start address >> 4).
//   K-major SWIZZLE_128B: 8-row groups 1 KB apart; 16 features further: + 32 bytes; box: + 16 KB.
//   MN-major SWIZZLE_128B: K groups of 8 rows 1 KB apart, the next 64 features one box (16 KB) on;
//   16 rows further: + 2 KB.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
// 2^x of two values in the FMA pipes (the exponential unit does 16 a cycle and SM, and bounds these kernels
// where a head has 64 features).  x = n + f, n the nearest integer: adding 1.5 * 2^23 leaves n in the low
// bits, 2^f is a polynomial, 2^n is built from its bits (Cody and Waite's reduction; the coefficients are a
// Remez fit of the relative error on [-1/2, 1/2]: 2.7e-6 = 2^-18.5 with the fp32 evaluation, far below the
// 2^-8 (bf16) or 2^-11 (fp16) of the weights' rounding).  x <= 100; x <= -127, -infinity among it, gives exactly 0; NaN stays NaN.
__device__ __forceinline__ float2 ex2_fma(float2 x) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(-127.f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(-127.f));
    const float2 big = make_float2(12582912.f, 12582912.f), neg = make_float2(-12582912.f, -12582912.f);
    const float2 t = add2(x, big);
    const float2 n = add2(t, neg);
    const float2 f = fma2(n, make_float2(-1.f, -1.f), x);
    float2 p = fma2(f, make_float2(0.009570102207362652f, 0.009570102207362652f),
                    make_float2(0.05591785907745361f, 0.05591785907745361f));
    p = fma2(p, f, make_float2(0.240247443318367f, 0.240247443318367f));
    p = fma2(p, f, make_float2(0.6931217908859253f, 0.6931217908859253f));
    p = fma2(p, f, make_float2(0.9999992847442627f, 0.9999992847442627f));
    return mul2(p, make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + 0x3F800000u),
                               __uint_as_float((__float_as_uint(t.y) << 23) + 0x3F800000u)));
}
// 2^x of pair number `pair`: by the FMA pipes where its bit of MASK (of 8) is set.
template <uint32_t MASK>
__device__ __forceinline__ float2 ex2_pair(float2 x, int pair) {
    if ((MASK >> (pair & 7)) & 1u) return ex2_fma(x);
    return make_float2(ex2(x.x), ex2(x.y));
}

// The high halves of both descriptors are the same constant; the loops below only add to the low ones, and
// are unrolled: one thread issues all MMAs, and what it computes between two of them delays the second.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) { return (static_cast<uint64_t>(kDescHi) << 32) | lo; }
__device__ __forceinline__ uint32_t desc_k_lo(uint32_t start) { return (1u << 16) | (start >> 4); }
// D[128 x N] = A B^T over `steps` * 16 of DP features, both tiles K-major; A has 128 rows, B BN.
template <int DP, int BN = kTile>
__device__ __forceinline__ void mma_features(uint32_t d, uint32_t a, uint32_t b, int steps, uint32_t idesc) {
    const uint32_t la = desc_k_lo(a), lb = desc_k_lo(b);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        const uint32_t in = static_cast<uint32_t>(s & 3) * 32, box = static_cast<uint32_t>(s >> 2);
        if (s < steps)
            ptx::umma_f16(d, desc_of(la + ((box * kBoxBytes + in) >> 4)), desc_of(lb + ((box * BN * 128 + in) >> 4)), idesc,
                          s > 0);
    }
}
// D[128 x N] (+)= A[tmem, 128 x BN] B over the BN rows of tile b, steps [FROM, TO) of 16.  A's K elements lie in
// `HALVES` equal parts, GAP columns apart.
template <int BN, int GAP, int HALVES, int FROM = 0, int TO = BN / 16>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    constexpr int PER = BN / 16 / HALVES;
    const uint32_t lb = ((static_cast<uint32_t>(BN) * 128 >> 4) << 16) | (b >> 4);   // LBO: the next 64 features
#pragma unroll
    for (int s = FROM; s < TO; ++s)
        umma_f16_ts(d, a + (s / PER) * GAP + (s % PER) * 8, desc_of(lb + s * (2048 >> 4)), idesc, add || s > 0);
}
constexpr uint32_t kBMnMajor = 1u << 16;         // instruction descriptor: B is MN-major

// Rows [valid, BN) of a tile as zeros (all lanes of one warp): a row of another sequence would turn a
// weight of zero into NaN if it holds an infinity or NaN.
template <int BN = kTile>
__device__ __forceinline__ void zero_tail(uint8_t* tile, int boxes, int valid, int lane) {
    for (int b = 0; b < boxes; ++b)
        for (int i = valid * 8 + lane; i < BN * 8; i += 32)
            *reinterpret_cast<uint4*>(tile + b * (BN * 128) + i * 16) = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
    __syncwarp();
}

// ------------------------------------------------------------------------------------- forward
//
// A block takes NQ tiles of 128 query rows of one head and walks their keys in tiles of 128.  Warps:
// NQ warpgroups of softmax (thread = query row = TMEM lane), one warp of loads, one of MMAs.
//   S_i = Q_i K^T                      (SS product, fp32 in TMEM)
//   m, l running maximum and sum; P = exp2(c (S - m)) rounded to the I/O type, in TMEM
//   O_i += P V                         (A from TMEM)
// The maximum that P refers to moves only when the true one has grown by more than 2^8: until then
// P stays below 2^8, and the rescaling of O (a round trip through registers) is rarely needed.
//
// D > 64: two query tiles in a block, so that the tensor cores work on one while the other's softmax runs.  Bound by
// the tensor cores: 1430 TFLOP/s over long keys with all SMs filled; a causal call of few long sequences by its
// longest one (12 sequences of up to 4096: 85 us, of which about 60 are the steps of one block).
// D <= 64: one query tile and two blocks on an SM.  The products of a tile of 128 x 128 take 512 cycles, its
// exponentials 1024 in the exponential unit alone, and the steps of a tile (scores out of TMEM, maximum, exponentials,
// weights into TMEM) follow one another; two blocks overlap them to 1480 cycles.  784 tokens, 32 sequences, 8 heads:
// 98 us (413 TFLOP/s; tensor cores busy 27 %, instructions issued in 42 % of the cycles); 8192 tokens, 8 heads: 198 us
// (694).  Measured instead, for these two: tiles of 64 keys with 2, 3, 4 blocks on an SM 114, 102, 95 and 258, 282,
// 228 us; two threads a row with their maxima exchanged through shared memory 103 and 217.
template <int DP, int NQ>
struct Fwd {
    static constexpr int BOXES = DP / 64;
    static constexpr int TILE_BYTES = BOXES * kBoxBytes;
    // D <= 64: two blocks per SM, each with half of the TMEM and at most 113 KB of shared memory
    static constexpr int STAGES = NQ == 2 ? (227 * 1024 - 2048) / TILE_BYTES - NQ : 4;
    static constexpr int THREADS = NQ * 128 + 64;
    static constexpr int WARP_LOAD = NQ * 4, WARP_MMA = NQ * 4 + 1;
    // with room in TMEM, P gets columns of its own, and the scores of the next tile are computed while
    // this one's weights are
    static constexpr bool OWN_P = NQ * (128 + DP + 64) <= (NQ == 1 ? 256 : 512);
    static constexpr int TMEM_COLS = NQ == 1 ? 256 : 512;
    // Share of the exponentials in the FMA pipes, of 8 pairs.  D <= 64: us for a tile of 128 x 128 with two
    // blocks on an SM: none 0.84, 2 of 8 0.75, 3 of 8 0.80, 4 of 8 0.85.  D = 128, where the products take
    // twice as long: none 0.90, 2 of 8 0.94.
    static constexpr uint32_t EX2_FMA = DP == 64 ? 0x44 : 0;
    static constexpr size_t SMEM = 1024 + 512 + static_cast<size_t>(STAGES + NQ) * TILE_BYTES;
};

struct FwdParams {
    Params p;
    long long stop_after;    // test hook: the load warp stops after this many tiles; -1 off
};

template <class T, int DP, int NQ>
__global__ void __launch_bounds__(Fwd<DP, NQ>::THREADS, NQ == 2 ? 1 : 2)
    eqlin_attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                             const __grid_constant__ CUtensorMap mv, const __grid_constant__ FwdParams fp) {
    using F = Fwd<DP, NQ>;
    constexpr int ST = F::STAGES;
    const Params& p = fp.p;
    extern __shared__ uint8_t raw[];
    uint8_t* base = ptx::smem_align_1k(raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + (F::STAGES + NQ) * F::TILE_BYTES);
    Ctl* ctl = reinterpret_cast<Ctl*>(bars + 48);
    auto bar = [&](int i) { return ptx::smem_u32(bars + i); };
    // barriers: [0, ST) full, [ST, 2 ST) empty, then per query tile: q, s, p, o
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(ST + s); };
    auto q_full = [&](int i) { return bar(2 * ST + i); };
    auto s_full = [&](int i) { return bar(2 * ST + NQ + i); };
    auto p_full = [&](int i) { return bar(2 * ST + 2 * NQ + i); };
    auto o_full = [&](int i) { return bar(2 * ST + 3 * NQ + i); };
    auto s_read = [&](int i) { return bar(2 * ST + 4 * NQ + i); };
    auto p_half = [&](int i) { return bar(2 * ST + 5 * NQ + i); };   // the weights of the first 64 keys
    const uint32_t drained = bar(2 * ST + 6 * NQ);
    uint8_t* q_tile = base;
    uint8_t* ring = base + NQ * F::TILE_BYTES;

    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (uniform)
    if (threadIdx.x == 0) {
        ptx::prefetch_tmap(&mq);
        ptx::prefetch_tmap(&mk);
        ptx::prefetch_tmap(&mv);
        ctl->abort = 0;
        for (int s = 0; s < ST; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int i = 0; i < NQ; ++i) {
            ptx::mbar_init(q_full(i), 1);
            ptx::mbar_init(s_full(i), 1);
            ptx::mbar_init(p_full(i), 4);
            ptx::mbar_init(p_half(i), 4);
            ptx::mbar_init(o_full(i), 1);
            ptx::mbar_init(s_read(i), 4);
        }
        ptx::mbar_init(drained, 1);
        ptx::fence_mbar_init();
    }
    if (warp == F::WARP_MMA) {
        ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem_base), F::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::grid_dependency_wait();

    // Heads vary fastest; the slots of a causal call run backwards, so that the tiles with the most
    // keys start first.
    const int h = blockIdx.x % p.heads, hk = h / (p.heads / p.kv_heads);
    const int n_slots = gridDim.x / p.heads;
    const int slot = p.causal ? n_slots - 1 - blockIdx.x / p.heads : blockIdx.x / p.heads;
    const Tile t = find_tile<NQ * kTile>(p.q_offsets, p.sequences, p.q_rows, slot);
    const Rows kr = other_rows(p, t, p.k_offsets, p.k_rows);
    const int r0 = t.tile * NQ * kTile;
    int count[NQ], n = 0;     // key tiles of each query tile
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int rows = t.tile < 0 ? 0 : min(kTile, t.own.len - r0 - i * kTile);
        count[i] = rows <= 0 ? 0
                             : (keys_seen(r0 + i * kTile + rows - 1, t.own.len, kr.len, p.causal) + kTile - 1) / kTile;
        n = max(n, count[i]);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    // only now: a dependent block that took this SM's TMEM first would wait for this grid, and this
    // block for the TMEM
    ptx::grid_launch_dependents();
    const uint32_t tmem = ctl->tmem_base;
    auto t_s = [&](int i) { return tmem + i * 128; };
    auto t_o = [&](int i) { return tmem + NQ * 128 + i * DP; };
    auto t_p = [&](int i) { return F::OWN_P ? tmem + NQ * (128 + DP) + i * 64 : t_s(i); };

    if (warp == F::WARP_LOAD) {
        if (lane == 0 && n > 0) {
            long long issued = 0;
            bool ok = true;
            auto load = [&](const CUtensorMap* m, uint8_t* dst, int head, int row, uint32_t b) {
                ptx::mbar_arrive_expect_tx(b, F::TILE_BYTES);
                for (int x = 0; x < F::BOXES; ++x)
                    tma_load_3d(ptx::smem_u32(dst) + x * kBoxBytes, m, x * 64, head, row, b);
            };
            for (int i = 0; i < NQ; ++i)
                if (count[i] > 0) load(&mq, q_tile + i * F::TILE_BYTES, h, t.own.start + r0 + i * kTile, q_full(i));
            for (int u = 0; ok && u < 2 * n; ++u) {      // K_0, V_0, K_1, V_1, ...
                const int s = u % ST;
                if (u >= ST && !wait_bounded(empty(s), ((u / ST) & 1) ^ 1, ctl, p.timeout_ns)) break;
                if (issued == fp.stop_after) break;
                load(u & 1 ? &mv : &mk, ring + s * F::TILE_BYTES, hk, kr.start + (u >> 1) * kTile, full(s));
                ++issued;
            }
            // every copy must land before the block's shared memory is given up
            for (int i = 0; i < NQ; ++i)
                if (count[i] > 0) drain_wait(q_full(i), 0, p.timeout_ns);
            for (int s = 0; s < ST; ++s) {
                const long long times = issued > s ? (issued - s + ST - 1) / ST : 0;
                if (times > 0) drain_wait(full(s), static_cast<uint32_t>((times - 1) & 1), p.timeout_ns);
            }
        }
    } else if (warp == F::WARP_MMA) {
        if (n > 0) {
            const uint32_t id_s = idesc_f16kind_f32(128, 128, Io16<T>::kUmmaFormat, false);
            const uint32_t id_o = idesc_f16kind_f32(128, (p.D + 15) / 16 * 16, Io16<T>::kUmmaFormat, false) | kBMnMajor;
            const int steps = (p.D + 15) / 16;
            bool ok = true;
            // ring position of a tile of keys (from 0) or values (from 1); both move on by two
            struct At {
                int s;
                uint32_t ph;
                __device__ void next() {
                    s += 2;
                    if (s >= ST) {
                        s -= ST;
                        ph ^= 1;
                    }
                }
            };
            At ks = {0, 0}, vs = {1 % ST, 1 / ST};
            const uint32_t ring32 = ptx::smem_u32(ring), q32 = ptx::smem_u32(q_tile);
            auto wait_stage = [&](const At& a) { return wait_warp(full(a.s), a.ph, ctl, p.timeout_ns); };
            auto scores = [&](int i) {
                if (elect_one()) {
                    mma_features<DP>(t_s(i), q32 + i * F::TILE_BYTES, ring32 + ks.s * F::TILE_BYTES, steps, id_s);
                    ptx::umma_commit(s_full(i));
                }
                __syncwarp();
            };
            ok = wait_stage(ks);
#pragma unroll
            for (int i = 0; i < NQ; ++i)
                if (ok && count[i] > 0) {
                    ok = wait_warp(q_full(i), 0, ctl, p.timeout_ns);
                    ptx::tc_fence_after();
                    if (ok) scores(i);
                }
            if (ok && elect_one()) ptx::umma_commit(empty(ks.s));
            ks.next();
            for (int j = 0; ok && j < n; ++j) {
                bool have_v = false, have_k = false;
                // the next scores of tile i: its S is free once it has been read (or, where P lies over
                // it, once the product that reads P has been issued: MMAs of one thread run in order)
                auto next_scores = [&](int i) {
                    if (!have_k) {
                        have_k = true;
                        if (!wait_stage(ks)) return false;
                    }
                    if (F::OWN_P && !wait_warp(s_read(i), j & 1, ctl, p.timeout_ns)) return false;
                    ptx::tc_fence_after();
                    scores(i);
                    return true;
                };
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    if (!ok || j >= count[i]) continue;
                    if (F::OWN_P && j + 1 < count[i] && !(ok = next_scores(i))) break;
                    if (!have_v) {
                        have_v = true;
                        if (!(ok = wait_stage(vs))) break;
                        const int valid = kr.len - j * kTile;
                        if (valid < kTile) zero_tail(ring + vs.s * F::TILE_BYTES, F::BOXES, valid, lane);
                    }
                    // the product with the first half of the weights runs while the second is computed
                    if (!(ok = wait_warp(p_half(i), j & 1, ctl, p.timeout_ns))) break;
                    ptx::tc_fence_after();
                    if (elect_one()) mma_rows<kTile, 0, 1, 0, 4>(t_o(i), t_p(i), ring32 + vs.s * F::TILE_BYTES, id_o, j > 0);
                    __syncwarp();
                    if (!(ok = wait_warp(p_full(i), j & 1, ctl, p.timeout_ns))) break;
                    ptx::tc_fence_after();
                    if (elect_one()) {
                        mma_rows<kTile, 0, 1, 4, 8>(t_o(i), t_p(i), ring32 + vs.s * F::TILE_BYTES, id_o, j > 0);
                        ptx::umma_commit(o_full(i));
                    }
                    __syncwarp();
                    if (!F::OWN_P && j + 1 < count[i] && !(ok = next_scores(i))) break;
                }
                if (ok && elect_one()) {
                    ptx::umma_commit(empty(vs.s));
                    if (j + 1 < n) ptx::umma_commit(empty(ks.s));
                }
                vs.next();
                ks.next();
            }
            // every MMA, and every arrival that one owes a barrier, before shared memory and TMEM go
            if (elect_one()) {
                ptx::umma_commit(drained);
                drain_wait(drained, 0, p.timeout_ns);
            }
            __syncwarp();
        }
    } else {
        const int i = NQ == 1 ? 0 : warp >> 2;
        const int cnt = NQ == 1 ? count[0] : (i == 0 ? count[0] : count[NQ - 1]);
        const int row = r0 + i * kTile + (threadIdx.x & 127);      // row of the sequence
        const bool live = t.tile >= 0 && row < t.own.len;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = t_s(i) + lanes, to = t_o(i) + lanes, tp = t_p(i) + lanes;
        // keys this row sees
        const int seen = live ? keys_seen(row, t.own.len, kr.len, p.causal) : 0;
        // keys that every row of the tile sees: tiles below need no mask
        const int seen_all = p.causal ? keys_seen(r0 + i * kTile, t.own.len, kr.len, 1) : kr.len;
        const float c2 = p.scale * kLog2e;
        float top = -INFINITY, sum = 0.f;
        bool ok = true;
        // A warp whose 32 rows all lie past the sequence's end only keeps the barriers' count: what its lanes of P
        // and O hold goes nowhere.
        const bool idle = t.tile < 0 || r0 + i * kTile + (warp & 3) * 32 >= t.own.len;
        for (int j = 0; j < cnt; ++j) {
            if (!(ok = wait_warp(s_full(i), j & 1, ctl, p.timeout_ns))) break;
            if (idle) {
                // never a phase ahead of the other warps: the weights of the tile before have all arrived
                if (j > 0 && !(ok = wait_warp(o_full(i), (j - 1) & 1, ctl, p.timeout_ns))) break;
                if (F::OWN_P) arrive_warp(s_read(i), lane);
                arrive_warp(p_half(i), lane);
                arrive_warp(p_full(i), lane);
                continue;
            }
            ptx::tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b<32>(ts + c * 32, s[c]);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c) ptx::tmem_regs_ready(s[c]);
            if (F::OWN_P) {
                ptx::tc_fence_before();
                arrive_warp(s_read(i), lane);
            }
            if ((j + 1) * kTile > seen_all) {
                const int n_seen = seen - j * kTile;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e >= n_seen) s[c][e] = 0xFF800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 2)
#pragma unroll
                for (int c = 0; c < 4; ++c) mx[c] = max3(mx[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
            const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            bool move = (m - top) * c2 > 8.f;                       // also the first finite maximum
            if (j == 0) {
                top = m;
            } else if (__any_sync(0xFFFFFFFFu, move)) {
                // O must be at rest: the product of the tile before is done
                if (!(ok = wait_warp(o_full(i), (j - 1) & 1, ctl, p.timeout_ns))) break;
                ptx::tc_fence_after();
                const float fade = move ? ex2((top - m) * c2) : 1.f;   // 0 while top is -infinity
                if (move) top = m;
                sum *= fade;
                for (int c = 0; c < p.D; c += 16) {
                    uint32_t o[16];
                    ptx::tmem_ld_32x32b<16>(to + c, o);
                    ptx::tmem_wait_ld();
                    ptx::tmem_regs_ready(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fade);
                    tmem_st16(to + c, o);
                }
            }
            const float off = top == -INFINITY ? 0.f : -top * c2;
            const float2 c22 = make_float2(c2, c2), off2 = make_float2(off, off);
            float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float2 a = fma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), c22, off2);
                    a = ex2_pair<F::EX2_FMA>(a, e >> 1);
                    part[(e >> 1) & 1] = add2(part[(e >> 1) & 1], a);
                    w[e >> 1] = Io16<T>::pack(a.x, a.y);
                }
                // P of the tile before has been read
                if (F::OWN_P && c == 0 && j > 0 && !(ok = wait_warp(o_full(i), (j - 1) & 1, ctl, p.timeout_ns))) break;
                tmem_st16(tp + c * 16, w);
                if (c == 1) {
                    tmem_wait_st();
                    ptx::tc_fence_before();
                    arrive_warp(p_half(i), lane);
                }
            }
            if (!ok) break;
            sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
            tmem_wait_st();
            ptx::tc_fence_before();
            arrive_warp(p_full(i), lane);
        }
        if (ok && cnt > 0) ok = wait_warp(o_full(i), (cnt - 1) & 1, ctl, p.timeout_ns);
        if (ok && t.tile >= 0) {
            ptx::tc_fence_after();
            const float inv = sum == 0.f ? 0.f : 1.f / sum;        // a row that sees no key
            const long long at = static_cast<long long>(t.own.start) + row;
            if (live && p.lse)
                p.lse[static_cast<long long>(h) * p.q_rows + at] =
                    sum == 0.f ? -INFINITY : fmaf(top * p.scale, 1.f, logf(sum));
            T* out = static_cast<T*>(p.out) + at * p.o_stride + static_cast<long long>(h) * p.D;
            for (int c = 0; c < p.D; c += 16) {
                uint32_t o[16] = {};
                if (cnt > 0) {
                    ptx::tmem_ld_32x32b<16>(to + c, o);
                    ptx::tmem_wait_ld();
                    ptx::tmem_regs_ready(o);
                }
                if (!live) continue;
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    if (c + e >= p.D) break;
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = Io16<T>::pack(__uint_as_float(o[e + 2 * k]) * inv, __uint_as_float(o[e + 2 * k + 1]) * inv);
                    *reinterpret_cast<uint4*>(out + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        ptx::tc_fence_before();
    }
    __syncthreads();
    if (warp == F::WARP_MMA) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, F::TMEM_COLS);
    }
}

}  // namespace tc
}  // namespace attn
}  // namespace eqlin
