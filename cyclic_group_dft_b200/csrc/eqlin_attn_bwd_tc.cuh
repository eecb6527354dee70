// eqlin_attn_bwd_tc.cuh -- gradients of 16-bit attention on the tcgen05 tensor cores.
//
// Two kernels, each with its sums in TMEM and without atomics, so that results do not vary:
//   dk, dv: a block holds 128 keys of one key head and walks the queries of its group's heads:
//       S^T = K Q^T,  dP^T = V dO^T,  P^T = exp2(c S^T - lse),  dS^T = P^T (dP^T - delta)
//       dV += P^T dO,  dK += dS^T Q           (A = P^T, dS^T from TMEM)
//   dq: a block holds 128 queries of one head and walks their keys:
//       S = Q K^T,  dP = dO V^T,  dS = P (dP - delta),  dQ += dS K
// Computing S and dP twice costs two more products than one kernel would (7 for 5), and saves the
// atomics or the fp32 copy of dq that one kernel needs.
// Warps: two warpgroups of 128 threads for the elementwise work (thread = TMEM lane; each warpgroup
// takes half of the columns, and its words of the A operand lie at the start of them), one warp of loads, one of MMAs.
//
// Bound by the chain of each tile (scores, weights, products), which the other tiles in flight overlap in part.  8192
// tokens: 6 heads of 128 features 584 us (880 TFLOP/s counting 5 products), 8 heads of 64 542 us (633); 784 tokens, 32
// sequences, 8 heads of 64: 240 us, tensor cores busy 36 to 38 %, instructions issued in 40 to 42 % of the cycles.
#pragma once

#include "eqlin_attn_tc.cuh"

namespace eqlin {
namespace attn {
namespace tc {

// BN: rows of a tile of the side that is walked.  For heads of up to 64 features it is 64: then a block needs
// half of the TMEM, and the chain of products and elementwise work of one block on an SM fills the gaps of the
// other's (784 tokens, 32 sequences, 8 heads: 239 us; one block of four warpgroups with BN = 128: 342).
template <int DP>
struct Bwd {
    static constexpr int BN = DP;
    static constexpr int HB = BN / 2;                    // columns of a warpgroup
    static constexpr int BOXES = DP / 64;
    static constexpr int OWN_BYTES = BOXES * kBoxBytes;  // 128 rows
    static constexpr int WALK_BYTES = BOXES * BN * 128;
    static constexpr int LOAD_ROWS = BN;                 // rows of a TMA box, for both sides
    static constexpr int STAGES = DP == 64 ? 8 : 5;
    static constexpr int TMEM_COLS = DP == 64 ? 256 : 512;
    static constexpr int BLOCKS = DP == 64 ? 2 : 1;
    static constexpr int THREADS = 256 + 64;
    static constexpr int WARP_LOAD = 8, WARP_MMA = 9;
    static constexpr int ROW_BUFS = STAGES / 2;          // of lse and delta, which come with dO
    static constexpr size_t SMEM =
        static_cast<size_t>(2) * OWN_BYTES + STAGES * WALK_BYTES + ROW_BUFS * 2 * BN * sizeof(float) + 256;
    static_assert(SMEM <= 232448 / BLOCKS, "shared memory");
};

struct BwdParams {
    Params p;
    long long stop_after;    // test hook, as in FwdParams
};

// Position in the ring: one step of the order in which its tiles are loaded.
template <int ST>
struct RingAt {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == ST) {
            s = 0;
            ph ^= 1;
        }
    }
};
// The walked query tiles in order: tiles [begin, end) of each head of a group.  Counted, not divided: the
// divisions of a flat index cost more than the waits that they stood before.
struct WalkAt {
    int tile, head, begin, end;
    __device__ __forceinline__ void next() {
        if (++tile == end) {
            tile = begin;
            ++head;
        }
    }
};

// 128 rows x D features of an fp32 accumulator in TMEM, times `mul`, to the rows of an output.
template <class T>
__device__ __forceinline__ void store_accumulator(uint32_t taddr, bool filled, bool live, T* out, int D, float mul) {
    for (int c = 0; c < D; c += 16) {
        uint32_t o[16] = {};
        if (filled) {
            ptx::tmem_ld_32x32b<16>(taddr + c, o);
            ptx::tmem_wait_ld();
            ptx::tmem_regs_ready(o);
        }
        if (!live) continue;
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
            if (c + e >= D) break;
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = Io16<T>::pack(__uint_as_float(o[e + 2 * k]) * mul, __uint_as_float(o[e + 2 * k + 1]) * mul);
            *reinterpret_cast<uint4*>(out + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// What the kernels below read of each query row: lse in units of log2 (less the lift of p) and delta = do . o, as
// [head][slot][lse 128, delta 128] with the slots of find_tile<128>, so that a tile's values are one aligned piece.
// A row that sees no key, or is past its sequence's end, gets lse = +infinity: weights of zero.  Both tensors are
// read once; bound by memory.
// fp16 (kLifted): for p <= 1, |ds_ij| <= |do_i| |v_j| + |delta_i|, by which ds can be lifted.  So each warp also leaves
// the largest |do_i| and |delta_i| of its rows ([head][slot][8][2]); the kernel for dk and dv adds those of |v_j| for
// the one for dq ([key head][slot][4]).  Infinite ones are left out: no exponent helps their products.
template <class T>
__global__ void __launch_bounds__(256) eqlin_attn_stats_kernel(const Params p) {
    using V = Vec<T, 8>;
    constexpr bool LIFT = kLifted<T>;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int h = blockIdx.x % p.heads, slot = blockIdx.x / p.heads, n_slots = gridDim.x / p.heads;
    const Tile t = find_tile<kTile>(p.q_offsets, p.sequences, p.q_rows, slot);
    if (t.tile < 0) return;
    const int r0 = t.tile * kTile, n = min(kTile, t.own.len - r0);
    const int lanes = p.D <= 64 ? 8 : 16;                // threads of a row
    const int lane = threadIdx.x & (lanes - 1), rows = 256 / lanes;
    const long long first = static_cast<long long>(t.own.start) + r0, tile = static_cast<long long>(h) * n_slots + slot;
    float* out = p.delta + tile * 2 * kTile;
    const bool in = lane * 8 < p.D;
    const T* a = static_cast<const T*>(p.dout) + first * p.do_stride + static_cast<long long>(h) * p.D + lane * 8;
    const T* b = static_cast<const T*>(p.o) + first * p.o_stride + static_cast<long long>(h) * p.D + lane * 8;
    float most = 0.f;                                    // of |delta| in the first thread of a row, of |do|^2 in another
#pragma unroll 4
    for (int r = threadIdx.x / lanes; r < kTile; r += rows) {
        float sum = 0.f, norm = 0.f;
        if (in && r < n) {
            float x[8], y[8];
            V::unpack(V::load(a + r * p.do_stride), x);
            V::unpack(V::load(b + r * p.o_stride), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum = fmaf(x[e], y[e], sum);
                if (LIFT) norm = fmaf(x[e], x[e], norm);
            }
        }
        if (LIFT) {   // half of the row's threads go on with one of the sums, half with the other
            const bool upper = lane & (lanes >> 1);
            const float other = __shfl_xor_sync(0xFFFFFFFFu, upper ? sum : norm, lanes >> 1);
            sum = (upper ? norm : sum) + other;
        }
        for (int o = LIFT ? lanes >> 2 : lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (LIFT && fabsf(sum) < INFINITY) most = fmaxf(most, fabsf(sum));
        if (lane == 0) {
            const float l = r < n ? p.lse[static_cast<long long>(h) * p.q_rows + first + r] : -INFINITY;
            out[r] = l == -INFINITY ? INFINITY : fmaf(l, kLog2e, -kLiftOf<T>);
            out[kTile + r] = sum;
        }
    }
    if (LIFT) {
        for (int o = lanes; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        float* to = p.do_most + (tile * 8 + (threadIdx.x >> 5)) * 2;
        if ((threadIdx.x & 31) == 0) to[1] = most;
        if ((threadIdx.x & 31) == lanes >> 1) to[0] = sqrtf(most);
    }
}

// |x| of a row of a tile of fp16 in shared memory (features past the head's end are zeros), 0 where it is not finite.
template <int DP>
__device__ __forceinline__ float row_norm(const uint8_t* tile, int row) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 8; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(tile + (c >> 3) * kBoxBytes + row * 128 + (((c ^ row) & 7) << 4));
        for (const uint32_t w : {v.x, v.y, v.z, v.w}) {
            s0 = fmaf(Io16<__half>::lo(w), Io16<__half>::lo(w), s0);
            s1 = fmaf(Io16<__half>::hi(w), Io16<__half>::hi(w), s1);
        }
    }
    s0 = sqrtf(s0 + s1);
    return s0 < INFINITY ? s0 : 0.f;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// ------------------------------------------------------------------------------- dk and dv
template <class T, int DP>
__global__ void __launch_bounds__(Bwd<DP>::THREADS, Bwd<DP>::BLOCKS)
    eqlin_attn_dkv_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                             const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                             const __grid_constant__ BwdParams bp) {
    using B = Bwd<DP>;
    constexpr int ST = B::STAGES;
    const Params& p = bp.p;
    constexpr int BN = B::BN, HB = B::HB;
    extern __shared__ __align__(1024) uint8_t base[];
    float* rows = reinterpret_cast<float*>(base + 2 * B::OWN_BYTES + ST * B::WALK_BYTES);   // buffers: lse [BN], delta [BN]
    uint64_t* bars = reinterpret_cast<uint64_t*>(rows + B::ROW_BUFS * 2 * BN);
    Ctl* ctl = reinterpret_cast<Ctl*>(bars + 30);
    auto bar = [&](int i) { return ptx::smem_u32(bars + i); };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(ST + s); };
    const uint32_t fixed_full = bar(2 * ST), s_full = bar(2 * ST + 1), dp_full = bar(2 * ST + 2),
                   p_full = bar(2 * ST + 3), ds_full = bar(2 * ST + 4), done = bar(2 * ST + 5);
    uint8_t *k_tile = base, *v_tile = base + B::OWN_BYTES, *ring = base + 2 * B::OWN_BYTES;

    if (ptx::smem_u32(base) & 1023u) {   // the swizzled tiles rely on the declared alignment
        if (threadIdx.x == 0) atomicCAS(&g_status, 0, kErrMisaligned);
        return;
    }
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (uniform)
    if (threadIdx.x == 0) {
        for (const CUtensorMap* m : {&mq, &mk, &mv, &mdo}) ptx::prefetch_tmap(m);
        ctl->abort = 0;
        for (int s = 0; s < ST; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        ptx::mbar_init(fixed_full, 1);
        ptx::mbar_init(s_full, 1);
        ptx::mbar_init(dp_full, 1);
        ptx::mbar_init(p_full, 8);
        ptx::mbar_init(ds_full, 8);
        ptx::mbar_init(done, 1);
        ptx::fence_mbar_init();
    }
    if (warp == B::WARP_MMA) {
        ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem_base), B::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::grid_dependency_wait();
    const int hk = blockIdx.x % p.kv_heads, slot = blockIdx.x / p.kv_heads, group = p.heads / p.kv_heads;
    const Tile t = find_tile<kTile>(p.k_offsets, p.sequences, p.k_rows, slot);
    const Rows qr = other_rows(p, t, p.q_offsets, p.q_rows);
    const int r0 = t.tile * kTile;
    // query tiles: from the first that sees the first key of this tile
    const int begin = t.tile < 0 ? 0 : first_query(r0, qr.len, t.own.len, p.causal) / BN;
    const int per_head = t.tile < 0 ? 0 : max(0, (qr.len + BN - 1) / BN - begin);
    const int n = per_head * group;
    const long long q_slots = p.q_rows / kTile + p.sequences;
    // slot of the sequence's first query tile (see find_tile)
    const int q_slot = p.q_offsets ? qr.start / kTile + max(t.b, 0) : 0;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::grid_launch_dependents();   // after the allocation, as in the forward
    const uint32_t tmem = ctl->tmem_base;
    const uint32_t t_s = tmem, t_dp = tmem + BN, t_dv = tmem + 2 * BN, t_dk = tmem + 2 * BN + DP;

    if (warp == B::WARP_LOAD) {
        if (lane == 0 && n > 0) {
            long long issued = 0;
            auto load = [&](const CUtensorMap* m, uint8_t* dst, int rows, int head, int row, uint32_t b) {
                for (int x = 0; x < B::BOXES; ++x)
                    for (int r = 0; r < rows; r += B::LOAD_ROWS)
                        tma_load_3d(ptx::smem_u32(dst) + x * rows * 128 + r * 128, m, x * 64, head, row + r, b);
            };
            ptx::mbar_arrive_expect_tx(fixed_full, 2 * B::OWN_BYTES);
            load(&mk, k_tile, kTile, hk, t.own.start + r0, fixed_full);
            load(&mv, v_tile, kTile, hk, t.own.start + r0, fixed_full);
            RingAt<ST> at;
            WalkAt w = {begin, hk * group, begin, begin + per_head};
            for (int u = 0; u < 2 * n; ++u) {      // Q_0, dO_0, Q_1, dO_1, ...
                if (u >= ST && !wait_bounded(empty(at.s), at.ph ^ 1, ctl, p.timeout_ns)) break;
                if (issued == bp.stop_after) break;
                ptx::mbar_arrive_expect_tx(full(at.s), B::WALK_BYTES + (u & 1 ? 2 * BN * 4 : 0));
                load(u & 1 ? &mdo : &mq, ring + at.s * B::WALK_BYTES, BN, w.head, qr.start + w.tile * BN, full(at.s));
                if (u & 1) {   // with dO: lse and delta of its rows
                    const int row = w.tile * BN;
                    const float* src = p.delta + (w.head * q_slots + q_slot + row / kTile) * 2 * kTile + row % kTile;
                    const uint32_t dst = ptx::smem_u32(rows + ((u >> 1) % B::ROW_BUFS) * 2 * BN);
                    ptx::bulk_load(dst, src, BN * 4, full(at.s));
                    ptx::bulk_load(dst + BN * 4, src + kTile, BN * 4, full(at.s));
                }
                ++issued;
                at.next();
                if (u & 1) w.next();
            }
            drain_wait(fixed_full, 0, p.timeout_ns);
            for (int s = 0; s < ST; ++s) {
                const long long times = issued > s ? (issued - s + ST - 1) / ST : 0;
                if (times > 0) drain_wait(full(s), static_cast<uint32_t>((times - 1) & 1), p.timeout_ns);
            }
        }
    } else if (warp == B::WARP_MMA) {
        if (n > 0) {
            const uint32_t id_s = idesc_f16kind_f32(128, BN, Io16<T>::kUmmaFormat, false);
            const uint32_t id_o = idesc_f16kind_f32(128, (p.D + 15) / 16 * 16, Io16<T>::kUmmaFormat, false) | kBMnMajor;
            const int steps = (p.D + 15) / 16;
            const uint32_t ring32 = ptx::smem_u32(ring), k32 = ptx::smem_u32(k_tile), v32 = ptx::smem_u32(v_tile);
            RingAt<ST> at;
            WalkAt w = {begin, 0, begin, begin + per_head};
            // the ring's next tile, with zeros for the rows past the sequence's end; its stage, or -1
            auto take = [&](bool last_of_pair) {
                if (!wait_warp(full(at.s), at.ph, ctl, p.timeout_ns)) return -1;
                const int valid = qr.len - w.tile * BN;
                if (valid < BN) zero_tail<BN>(ring + at.s * B::WALK_BYTES, B::BOXES, valid, lane);
                const int s = at.s;
                at.next();
                if (last_of_pair) w.next();
                return s;
            };
            auto product = [&](uint32_t d, uint32_t fixed, int s, uint32_t b) {
                if (elect_one()) {
                    mma_features<DP, BN>(d, fixed, ring32 + s * B::WALK_BYTES, steps, id_s);
                    ptx::umma_commit(b);
                }
                __syncwarp();
            };
            int sq = -1, sdo = -1, sq_next = -1;
            bool ok = wait_warp(fixed_full, 0, ctl, p.timeout_ns) && (sq = take(false)) >= 0;
            if (ok) product(t_s, k32, sq, s_full);
            ok = ok && (sdo = take(true)) >= 0;
            if (ok) product(t_dp, v32, sdo, dp_full);
            for (int j = 0; ok && j < n; ++j) {
                if (!(ok = wait_warp(p_full, j & 1, ctl, p.timeout_ns))) break;
                ptx::tc_fence_after();
                if (elect_one()) mma_rows<BN, HB, 2>(t_dv, t_s, ring32 + sdo * B::WALK_BYTES, id_o, j > 0);
                __syncwarp();
                // MMAs of one thread run in order: S^T is written after P^T has been read out of it
                if (j + 1 < n) {
                    if (!(ok = (sq_next = take(false)) >= 0)) break;
                    product(t_s, k32, sq_next, s_full);
                }
                if (!(ok = wait_warp(ds_full, j & 1, ctl, p.timeout_ns))) break;
                ptx::tc_fence_after();
                if (elect_one()) {
                    mma_rows<BN, HB, 2>(t_dk, t_dp, ring32 + sq * B::WALK_BYTES, id_o, j > 0);
                    ptx::umma_commit(empty(sq));
                    ptx::umma_commit(empty(sdo));
                }
                __syncwarp();
                sq = sq_next;
                if (j + 1 < n) {
                    if (!(ok = (sdo = take(true)) >= 0)) break;
                    product(t_dp, v32, sdo, dp_full);
                }
            }
            if (elect_one()) {
                ptx::umma_commit(done);
                drain_wait(done, 0, p.timeout_ns);
            }
            __syncwarp();
        }
    } else {
        const int half = warp >> 2, tid = threadIdx.x;
        const int row = r0 + (tid & 127);                          // key of the sequence
        const bool live = t.tile >= 0 && row < t.own.len;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = t_s + lanes + half * HB, tdp = t_dp + lanes + half * HB;
        const float c2 = p.scale * kLog2e;
        bool ok = true;
        // a warp whose 32 keys all lie past the end only keeps the barriers' count
        const bool idle = t.tile < 0 || r0 + (warp & 3) * 32 >= t.own.len;
        // fp16: ds of this key lifted by its own |v| and the largest of the rows that the block walks
        int lift = 0;
        float own_v = 0.f;
        if constexpr (kLifted<T>) {
            if (!idle && n > 0) {
                const int first = begin * BN / kTile, values = ((qr.len + kTile - 1) / kTile - first) * 8;
                float a = 0.f, d = 0.f;
                for (int g = 0; g < group; ++g) {
                    const float2* most = reinterpret_cast<const float2*>(p.do_most) +
                                         ((static_cast<long long>(hk) * group + g) * q_slots + q_slot + first) * 8;
                    for (int i = lane; i < values; i += 32) {
                        const float2 m = most[i];
                        a = fmaxf(a, m.x);
                        d = fmaxf(d, m.y);
                    }
                }
                a = warp_max(a);
                d = warp_max(d);
                ok = wait_warp(fixed_full, 0, ctl, p.timeout_ns);
                if (ok && live) own_v = row_norm<DP>(v_tile, tid & 127);
                lift = lift_of(fmaf(a, own_v, d));
            }
        }
        for (int j = 0; ok && idle && j < n; ++j) {
            if (!(ok = wait_warp(s_full, j & 1, ctl, p.timeout_ns))) break;
            arrive_warp(p_full, lane);
            if (!(ok = wait_warp(dp_full, j & 1, ctl, p.timeout_ns))) break;
            arrive_warp(ds_full, lane);
        }
        WalkAt cw = {begin, 0, begin, begin + per_head};
        RingAt<ST> at;
        at.next();                                                 // dO_0
        const float up = power_of_two(lift - kLiftP);                  // p is lifted already
        for (int j = 0; ok && !idle && j < n; ++j) {
            const float* rj = rows + (j % B::ROW_BUFS) * 2 * BN;
            if (!(ok = wait_warp(full(at.s), at.ph, ctl, p.timeout_ns))) break;
            at.next();
            at.next();
            if (!(ok = wait_warp(s_full, j & 1, ctl, p.timeout_ns))) break;
            ptx::tc_fence_after();
            uint32_t s[HB / 32][32];
#pragma unroll
            for (int c = 0; c < HB / 32; ++c) ptx::tmem_ld_32x32b<32>(ts + c * 32, s[c]);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < HB / 32; ++c) ptx::tmem_regs_ready(s[c]);
            const int q0 = cw.tile * BN;
            cw.next();
            if (p.causal && static_cast<long long>(r0) + kTile - 1 > static_cast<long long>(q0) + t.own.len - qr.len) {
                // key `row` is seen by queries from row - (keys - queries) on
                const long long first = static_cast<long long>(row) - (t.own.len - qr.len) - q0 - half * HB;
#pragma unroll
                for (int c = 0; c < HB / 32; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e < first) s[c][e] = 0xFF800000u;
            }
#pragma unroll
            for (int c = 0; c < HB / 32; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(rj + half * HB + c * 32 + e);
                    const float2 a = fma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                          make_float2(c2, c2), make_float2(-l.x, -l.y));
                    const float2 b = fma2(make_float2(__uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3])),
                                          make_float2(c2, c2), make_float2(-l.z, -l.w));
                    const float v[4] = {ex2(a.x), ex2(a.y), ex2(b.x), ex2(b.y)};
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[c][e + k] = __float_as_uint(kLifted<T> ? v[k] * up : v[k]);
                    w[e >> 1] = Io16<T>::pack(v[0], v[1]);
                    w[(e >> 1) + 1] = Io16<T>::pack(v[2], v[3]);
                }
                tmem_st16(ts + c * 16, w);
            }
            tmem_wait_st();
            ptx::tc_fence_before();
            arrive_warp(p_full, lane);
            if (!(ok = wait_warp(dp_full, j & 1, ctl, p.timeout_ns))) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int c = 0; c < HB / 32; ++c) {
                uint32_t d[32], w[16];
                ptx::tmem_ld_32x32b<32>(tdp + c * 32, d);
                ptx::tmem_wait_ld();
                ptx::tmem_regs_ready(d);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(rj + BN + half * HB + c * 32 + e);
                    const float2 a = mul2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                          add2(make_float2(__uint_as_float(d[e]), __uint_as_float(d[e + 1])),
                                               make_float2(-l.x, -l.y)));
                    const float2 b = mul2(make_float2(__uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3])),
                                          add2(make_float2(__uint_as_float(d[e + 2]), __uint_as_float(d[e + 3])),
                                               make_float2(-l.z, -l.w)));
                    w[e >> 1] = Io16<T>::pack(a.x, a.y);
                    w[(e >> 1) + 1] = Io16<T>::pack(b.x, b.y);
                }
                // words over columns that this thread has read
                tmem_st16(tdp + c * 16, w);
            }
            tmem_wait_st();
            ptx::tc_fence_before();
            arrive_warp(ds_full, lane);
        }
        if (kLifted<T> && half == 0 && n > 0) {   // the warps' largest |v|, for dq
            own_v = warp_max(own_v);
            if (lane == 0) p.v_most[(static_cast<long long>(hk) * (gridDim.x / p.kv_heads) + slot) * 4 + warp] = own_v;
        }
        if (ok && n > 0) ok = wait_warp(done, 0, ctl, p.timeout_ns);
        if (ok && t.tile >= 0) {
            ptx::tc_fence_after();
            const long long at = static_cast<long long>(t.own.start) + row, col = static_cast<long long>(hk) * p.D;
            if (half) store_accumulator<T>(t_dk + lanes, n > 0, live, static_cast<T*>(p.dk) + at * p.dk_stride + col, p.D,
                                           kLifted<T> ? p.scale * power_of_two(-lift) : p.scale);
            else store_accumulator<T>(t_dv + lanes, n > 0, live, static_cast<T*>(p.dv) + at * p.dv_stride + col, p.D,
                                      kLifted<T> ? power_of_two(-kLiftP) : 1.f);
        }
        ptx::tc_fence_before();
    }
    __syncthreads();
    if (warp == B::WARP_MMA) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, B::TMEM_COLS);
    }
}

// ------------------------------------------------------------------------------------- dq
template <class T, int DP>
__global__ void __launch_bounds__(Bwd<DP>::THREADS, Bwd<DP>::BLOCKS)
    eqlin_attn_dq_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                            const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                            const __grid_constant__ BwdParams bp) {
    using B = Bwd<DP>;
    constexpr int ST = B::STAGES;
    const Params& p = bp.p;
    constexpr int BN = B::BN, HB = B::HB;
    extern __shared__ __align__(1024) uint8_t base[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + 2 * B::OWN_BYTES + ST * B::WALK_BYTES);
    Ctl* ctl = reinterpret_cast<Ctl*>(bars + 30);
    auto bar = [&](int i) { return ptx::smem_u32(bars + i); };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(ST + s); };
    const uint32_t fixed_full = bar(2 * ST), dp_full = bar(2 * ST + 1), ds_full = bar(2 * ST + 2), done = bar(2 * ST + 3);
    auto s_full = [&](int b) { return bar(2 * ST + 4 + b); };
    uint8_t *q_tile = base, *do_tile = base + B::OWN_BYTES, *ring = base + 2 * B::OWN_BYTES;

    if (ptx::smem_u32(base) & 1023u) {   // the swizzled tiles rely on the declared alignment
        if (threadIdx.x == 0) atomicCAS(&g_status, 0, kErrMisaligned);
        return;
    }
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (uniform)
    if (threadIdx.x == 0) {
        for (const CUtensorMap* m : {&mq, &mk, &mv, &mdo}) ptx::prefetch_tmap(m);
        ctl->abort = 0;
        for (int s = 0; s < ST; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        ptx::mbar_init(fixed_full, 1);
        ptx::mbar_init(dp_full, 1);
        ptx::mbar_init(ds_full, 8);
        ptx::mbar_init(done, 1);
        ptx::mbar_init(s_full(0), 1);
        ptx::mbar_init(s_full(1), 1);
        ptx::fence_mbar_init();
    }
    if (warp == B::WARP_MMA) {
        ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem_base), B::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::grid_dependency_wait();
    const int h = blockIdx.x % p.heads, hk = h / (p.heads / p.kv_heads);
    const int n_slots = gridDim.x / p.heads;
    const int slot = p.causal ? n_slots - 1 - blockIdx.x / p.heads : blockIdx.x / p.heads;
    const Tile t = find_tile<kTile>(p.q_offsets, p.sequences, p.q_rows, slot);
    const Rows kr = other_rows(p, t, p.k_offsets, p.k_rows);
    const int r0 = t.tile * kTile;
    const int n = t.tile < 0 ? 0
                             : (keys_seen(min(r0 + kTile, t.own.len) - 1, t.own.len, kr.len, p.causal) + BN - 1) / BN;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::grid_launch_dependents();   // after the allocation, as in the forward
    const uint32_t tmem = ctl->tmem_base;
    auto t_s = [&](int j) { return tmem + (j & 1) * BN; };
    const uint32_t t_dp = tmem + 2 * BN, t_dq = tmem + 3 * BN;

    if (warp == B::WARP_LOAD) {
        if (lane == 0 && n > 0) {
            long long issued = 0;
            auto load = [&](const CUtensorMap* m, uint8_t* dst, int rows, int head, int row, uint32_t b) {
                for (int x = 0; x < B::BOXES; ++x)
                    for (int r = 0; r < rows; r += B::LOAD_ROWS)
                        tma_load_3d(ptx::smem_u32(dst) + x * rows * 128 + r * 128, m, x * 64, head, row + r, b);
            };
            ptx::mbar_arrive_expect_tx(fixed_full, 2 * B::OWN_BYTES);
            load(&mq, q_tile, kTile, h, t.own.start + r0, fixed_full);
            load(&mdo, do_tile, kTile, h, t.own.start + r0, fixed_full);
            RingAt<ST> at;
            for (int u = 0; u < 2 * n; ++u) {      // K_0, V_0, K_1, V_1, ...
                if (u >= ST && !wait_bounded(empty(at.s), at.ph ^ 1, ctl, p.timeout_ns)) break;
                if (issued == bp.stop_after) break;
                ptx::mbar_arrive_expect_tx(full(at.s), B::WALK_BYTES);
                load(u & 1 ? &mv : &mk, ring + at.s * B::WALK_BYTES, BN, hk, kr.start + (u >> 1) * BN, full(at.s));
                ++issued;
                at.next();
            }
            drain_wait(fixed_full, 0, p.timeout_ns);
            for (int s = 0; s < ST; ++s) {
                const long long times = issued > s ? (issued - s + ST - 1) / ST : 0;
                if (times > 0) drain_wait(full(s), static_cast<uint32_t>((times - 1) & 1), p.timeout_ns);
            }
        }
    } else if (warp == B::WARP_MMA) {
        if (n > 0) {
            const uint32_t id_s = idesc_f16kind_f32(128, BN, Io16<T>::kUmmaFormat, false);
            const uint32_t id_o = idesc_f16kind_f32(128, (p.D + 15) / 16 * 16, Io16<T>::kUmmaFormat, false) | kBMnMajor;
            const int steps = (p.D + 15) / 16;
            const uint32_t ring32 = ptx::smem_u32(ring), q32 = ptx::smem_u32(q_tile), do32 = ptx::smem_u32(do_tile);
            // the ring positions of the next K (for the scores), V, and K (for dQ)
            RingAt<ST> ks, vs, ks_dq;
            vs.next();
            auto scores = [&](int j) {
                if (!wait_warp(full(ks.s), ks.ph, ctl, p.timeout_ns)) return false;
                const int valid = kr.len - j * BN;
                if (valid < BN) zero_tail<BN>(ring + ks.s * B::WALK_BYTES, B::BOXES, valid, lane);
                if (elect_one()) {
                    mma_features<DP, BN>(t_s(j), q32, ring32 + ks.s * B::WALK_BYTES, steps, id_s);
                    ptx::umma_commit(s_full(j & 1));
                }
                __syncwarp();
                ks.next();
                ks.next();
                return true;
            };
            auto dp = [&] {
                if (!wait_warp(full(vs.s), vs.ph, ctl, p.timeout_ns)) return false;
                if (elect_one()) {
                    mma_features<DP, BN>(t_dp, do32, ring32 + vs.s * B::WALK_BYTES, steps, id_s);
                    ptx::umma_commit(dp_full);
                    ptx::umma_commit(empty(vs.s));
                }
                __syncwarp();
                vs.next();
                vs.next();
                return true;
            };
            bool ok = wait_warp(fixed_full, 0, ctl, p.timeout_ns) && scores(0) && dp();
            if (ok && n > 1) ok = scores(1);
            for (int j = 0; ok && j < n; ++j) {
                // dS_j lies over S_j, and dP_j has been read
                if (!(ok = wait_warp(ds_full, j & 1, ctl, p.timeout_ns))) break;
                ptx::tc_fence_after();
                if (j + 1 < n && !(ok = dp())) break;
                if (elect_one()) {
                    mma_rows<BN, HB, 2>(t_dq, t_s(j), ring32 + ks_dq.s * B::WALK_BYTES, id_o, j > 0);
                    ptx::umma_commit(empty(ks_dq.s));
                }
                __syncwarp();
                ks_dq.next();
                ks_dq.next();
                // MMAs of one thread run in order: S_{j+2} is written after dS_j has been read
                if (j + 2 < n) ok = scores(j + 2);
            }
            if (elect_one()) {
                ptx::umma_commit(done);
                drain_wait(done, 0, p.timeout_ns);
            }
            __syncwarp();
        }
    } else {
        const int half = warp >> 2;
        const int row = r0 + (threadIdx.x & 127);                  // query of the sequence
        const bool live = t.tile >= 0 && row < t.own.len;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int seen = live ? keys_seen(row, t.own.len, kr.len, p.causal) : 0;
        const int seen_all = p.causal ? keys_seen(r0, t.own.len, kr.len, 1) : kr.len;
        const float c2 = p.scale * kLog2e;
        const long long at = static_cast<long long>(t.own.start) + row;
        float off = 0.f, delta = 0.f;
        if (live && seen > 0) {
            const float* stat = p.delta + (static_cast<long long>(h) * n_slots + slot) * 2 * kTile + (threadIdx.x & 127);
            off = -stat[0];
            delta = stat[kTile];
        }
        bool ok = true;
        // a warp whose 32 queries all lie past the end only keeps the barriers' count
        const bool idle = t.tile < 0 || r0 + (warp & 3) * 32 >= t.own.len;
        // fp16: ds of this query lifted by its own |do| and delta and the largest |v| of the keys that the block walks
        int lift = 0;
        if constexpr (kLifted<T>) {
            if (!idle && n > 0) {
                const long long k_slots = p.k_rows / kTile + p.sequences;
                const float* most = p.v_most + (hk * k_slots + (p.k_offsets ? kr.start / kTile + t.b : 0)) * 4;
                const int values = (n * BN + kTile - 1) / kTile * 4;
                float v = 0.f;
                for (int i = lane; i < values; i += 32) v = fmaxf(v, most[i]);
                v = warp_max(v);
                ok = wait_warp(fixed_full, 0, ctl, p.timeout_ns);
                if (ok) lift = lift_of(fmaf(row_norm<DP>(do_tile, threadIdx.x & 127), v, fabsf(delta)));
            }
        }
        const float up = power_of_two(lift - kLiftP), down = -delta * up;   // p is lifted already
        for (int j = 0; ok && idle && j < n; ++j) {
            if (!(ok = wait_warp(s_full(j & 1), (j >> 1) & 1, ctl, p.timeout_ns))) break;
            if (!(ok = wait_warp(dp_full, j & 1, ctl, p.timeout_ns))) break;
            arrive_warp(ds_full, lane);
        }
        for (int j = 0; ok && !idle && j < n; ++j) {
            const uint32_t ts = t_s(j) + lanes + half * HB, tdp = t_dp + lanes + half * HB;
            if (!(ok = wait_warp(s_full(j & 1), (j >> 1) & 1, ctl, p.timeout_ns))) break;
            ptx::tc_fence_after();
            uint32_t s[HB / 32][32];
#pragma unroll
            for (int c = 0; c < HB / 32; ++c) ptx::tmem_ld_32x32b<32>(ts + c * 32, s[c]);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < HB / 32; ++c) ptx::tmem_regs_ready(s[c]);
            const bool masked = (j + 1) * BN > seen_all;
            const int n_seen = seen - j * BN - half * HB;
            if (masked) {
#pragma unroll
                for (int c = 0; c < HB / 32; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e >= n_seen) s[c][e] = 0xFF800000u;
            }
#pragma unroll
            for (int c = 0; c < HB / 32; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 a = fma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                          make_float2(c2, c2), make_float2(off, off));
                    s[c][e] = __float_as_uint(ex2(a.x));
                    s[c][e + 1] = __float_as_uint(ex2(a.y));
                }
            if (!(ok = wait_warp(dp_full, j & 1, ctl, p.timeout_ns))) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int c = 0; c < HB / 32; ++c) {
                uint32_t d[32], w[16];
                ptx::tmem_ld_32x32b<32>(tdp + c * 32, d);
                ptx::tmem_wait_ld();
                ptx::tmem_regs_ready(d);
                if (masked) {       // rows of V past the end may hold anything
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e >= n_seen) d[e] = 0;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 dp = make_float2(__uint_as_float(d[e]), __uint_as_float(d[e + 1]));
                    const float2 a = mul2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                          kLifted<T> ? fma2(dp, make_float2(up, up), make_float2(down, down))
                                                     : add2(dp, make_float2(-delta, -delta)));
                    w[e >> 1] = Io16<T>::pack(a.x, a.y);
                }
                tmem_st16(ts + c * 16, w);
            }
            tmem_wait_st();
            ptx::tc_fence_before();
            arrive_warp(ds_full, lane);
        }
        if (ok && n > 0) ok = wait_warp(done, 0, ctl, p.timeout_ns);
        if (ok && t.tile >= 0 && half == 0) {
            ptx::tc_fence_after();
            store_accumulator<T>(t_dq + lanes, n > 0, live,
                                 static_cast<T*>(p.dq) + at * p.dq_stride + static_cast<long long>(h) * p.D, p.D,
                                 kLifted<T> ? p.scale * power_of_two(-lift) : p.scale);
        }
        ptx::tc_fence_before();
    }
    __syncthreads();
    if (warp == B::WARP_MMA) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, B::TMEM_COLS);
    }
}

}  // namespace tc
}  // namespace attn
}  // namespace eqlin
