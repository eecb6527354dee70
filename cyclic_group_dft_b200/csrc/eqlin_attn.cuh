// eqlin_attn.cuh -- what the attention kernels share: parameters, packed sequences and the
// kernel that prepares the gradients.
//
// For query row i and key row j of one sequence and one head (D features: channels times group
// elements, so a cyclic shift of the group axis of q and k leaves every product unchanged and
// a shift of v shifts the output):
//     s_ij = scale * q_i . k_j,   p_ij = exp(s_ij - lse_i) over the visible j,   o_i = sum_j p_ij v_j
// Causal: query i of Lq sees key j of Lk when j <= i + Lk - Lq (the last query sees every key).
// A row that sees no key has o = 0, lse = -infinity and zero gradients.
//     dv_j = sum_i p_ij do_i,  ds_ij = p_ij (do_i . v_j - delta_i),  delta_i = do_i . o_i
//     dq_i = scale * sum_j ds_ij k_j,   dk_j = scale * sum_i ds_ij q_i
// Query head h reads key/value head h / (heads / kv_heads); dk and dv of a shared head sum over
// its query heads inside one block, so no atomics are used and results do not vary.
#pragma once

#include <cstdint>
#include <type_traits>

#include "eqlin_vec.cuh"
#include "sm100_ptx.cuh"

namespace eqlin {
namespace attn {

struct Params {
    const void *q, *k, *v, *o, *dout;
    void *out, *dq, *dk, *dv;      // out: the forward's o
    float* lse;                    // [heads][q_rows], or NULL
    float* delta;                  // gradients: delta [heads][q_rows], or the tensor-core kernels' statistics
    float *do_most, *v_most;       // and, for fp16, what bounds ds (see eqlin_attn_stats_kernel)
    const int32_t *q_offsets, *k_offsets;   // [sequences + 1], or NULL: one sequence of all rows
    long long q_stride, k_stride, v_stride, o_stride, do_stride, dq_stride, dk_stride, dv_stride;
    int q_rows, k_rows, sequences, heads, kv_heads, D;
    int causal;
    float scale;
    int splits;                    // slices of the keys; above 1 a slice's o and lse go to
    float *part_o, *part_lse;      // [splits][heads][q_rows][D] and [splits][heads][q_rows]
    unsigned long long timeout_ns;
};

// Rows [start, start + len) of sequence b.  Offsets live in device memory, where the host cannot
// check them: they are clamped to the tensor's rows and to one another, so that bad ones give
// wrong sequences but no access outside the tensors.
struct Rows {
    int start, len;
};
__device__ __forceinline__ Rows sequence_rows(const int32_t* offsets, int b, int rows) {
    if (!offsets) return {0, rows};
    const int s = min(max(offsets[b], 0), rows);
    const int e = min(max(offsets[b + 1], s), rows);
    return {s, e - s};
}

// Blocks are given tiles of M consecutive rows of one sequence without knowing the lengths on the
// host.  Sequence b owns the slots [off[b] / M + b, off[b+1] / M + b + 1): at least as many as it has
// tiles, in order, and rows / M + sequences in all.  A slot past its sequence's last tile has none.
// The slot's sequence is the last b whose first slot is not past it.  Sequences of about one length put
// it near slot * sequences / slots: 32 lanes probe the offsets around there in one read.  Otherwise 32
// lanes probe at once over the whole range, in log32(sequences) reads.  Every lane of the warp must call
// it.  `mult` rows of a tile for each row of the tensor (packed heads).
struct Tile {
    int b;       // sequence
    int tile;    // tile within the sequence, or -1: none
    Rows own;    // the sequence's rows on this side
};
// LATER: the slots of tiles 1, 2, .. alone (see for_short_tiles).
template <int M, bool LATER = false>
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int sequences, int rows, int slot, int mult = 1) {
    Tile t;
    if (!offsets) {
        t.b = 0;
        t.own = {0, rows};
        t.tile = static_cast<long long>(slot) * M < static_cast<long long>(rows) * mult ? slot : -1;
        return t;
    }
    auto offset = [&](int b) { return min(max(offsets[b], 0), rows); };
    auto first_slot = [&](int off, int b) {   // mult is 1, or the product with it is small (a few packed rows)
        return static_cast<long long>(static_cast<unsigned long long>(off) * mult / M) + (LATER ? 1 : b);
    };
    const int lane = threadIdx.x & 31;
    const float slots = static_cast<float>(rows) * mult * (1.f / M) + (LATER ? 1 : sequences);
    const int guess = static_cast<int>(__fdividef(static_cast<float>(slot) * sequences, slots));
    const int base = max(0, min(guess - 15, sequences - 31));
    const int probe = base + lane;
    const int off = offset(min(probe, sequences));
    const unsigned m = __ballot_sync(0xFFFFFFFFu, probe < sequences && first_slot(off, probe) <= slot);
    const int in = m ? 31 - __clz(m) : 0;
    int start, end;
    if ((m & 1u) && in < 31 && (m == (2u << in) - 1u)) {
        // [base, base + in] begin at or before the slot, base + in + 1 does not or is past the last one
        t.b = base + in;
        start = __shfl_sync(0xFFFFFFFFu, off, in);
        end = max(start, __shfl_sync(0xFFFFFFFFu, off, in + 1));
    } else {
        int lo = 0, n = sequences;   // the answer lies in [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) / 32;
            const int at = lo + lane * step;
            const bool ok = lane * step < n && first_slot(offset(at), at) <= slot;
            const unsigned w = __ballot_sync(0xFFFFFFFFu, ok);
            const int last = w ? 31 - __clz(w) : 0;
            const int rest = n - last * step;
            lo += last * step;
            n = rest < step ? rest : step;
        }
        t.b = lo;
        start = offset(lo);
        end = max(start, offset(lo + 1));
    }
    t.own = {start, end - start};
    const long long tile = slot - first_slot(start, t.b) + (LATER ? 1 : 0);
    t.tile = tile >= (LATER ? 1 : 0) && tile * M < static_cast<long long>(t.own.len) * mult ? static_cast<int>(tile) : -1;
    return t;
}

// The other side's rows of the tile's sequence; without a further read where both sides share their offsets.
__device__ __forceinline__ Rows other_rows(const Params& p, const Tile& t, const int32_t* offsets, int rows) {
    return p.k_offsets == p.q_offsets && p.k_rows == p.q_rows ? t.own : sequence_rows(offsets, t.b, rows);
}

// Keys [0, n) that query rows up to `last` (within the sequence) may see.
__device__ __forceinline__ int keys_seen(int last, int q_len, int k_len, int causal) {
    if (!causal) return k_len;
    const long long n = static_cast<long long>(last) + 1 + k_len - q_len;
    return static_cast<int>(n < 0 ? 0 : (n < k_len ? n : k_len));
}
// First query row (within the sequence) that sees key `first`.
__device__ __forceinline__ int first_query(int first, int q_len, int k_len, int causal) {
    if (!causal) return 0;
    const long long i = static_cast<long long>(first) + q_len - k_len;
    return static_cast<int>(i < 0 ? 0 : i);
}

// The gradients round p and ds to the I/O type before their products.  fp16 loses what is below 2^-14 there and has
// nothing above 65504, so both are lifted by powers of two, which the outputs take back exactly: p <= 1 by 2^12, ds
// to below 2^13 by what its largest value, or a bound of it for p <= 1, allows (row by row, see the kernels).  That
// leaves room for p above 1, where scores of 10^7 and more leave exp(s - lse) no correct bit.  Without the lift, 784
// tokens with dO of 2^-14 and v of 2^-6 lost dq whole.  What it costs, against none: 4096 windows of 49, 3 heads of 128
// features 323 to 333 us; 784 tokens, 32 sequences, 8 heads of 64 238 to 255; 8192 tokens 571 to 592; 100 tokens, 300
// sequences 165 to 184; 64 queries, 128 keys, 64 sequences, 8 heads on 2 71 to 79.
template <class T>
constexpr bool kLifted = std::is_same<T, __half>::value;
constexpr int kLiftP = 12;
template <class T>
constexpr float kLiftOf = kLifted<T> ? static_cast<float>(kLiftP) : 0.f;
constexpr int kLiftMost = 92;
// The exponent e for values of up to `most`: most * 2^e < 2^13.  Infinite and vanishing ones get a finite e.
__device__ __forceinline__ int lift_of(float most) {
    const int e = static_cast<int>((__float_as_uint(most) >> 23) & 255u) - 127;
    return 12 - max(12 - kLiftMost, min(e, 80));
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23); }

// delta[h][i] = do_i . o_i in fp32: one warp per (row, 32 / lanes heads), reading both tensors
// once.  A head takes `lanes` = the power of two >= D / VEC lanes.
template <class T, int VEC>
__global__ void __launch_bounds__(256) eqlin_attn_delta_kernel(const Params p, int lanes) {
    using V = Vec<T, VEC>;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int per_block = 256 / lanes;
    const long long unit = static_cast<long long>(blockIdx.x) * per_block + threadIdx.x / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const bool live = unit < static_cast<long long>(p.q_rows) * p.heads;
    const int row = live ? static_cast<int>(unit / p.heads) : 0;
    const int h = live ? static_cast<int>(unit - static_cast<long long>(row) * p.heads) : 0;
    float s = 0.f;
    if (live && lane * VEC < p.D) {
        float a[VEC], b[VEC];
        V::unpack(V::load(static_cast<const T*>(p.dout) + row * p.do_stride + static_cast<long long>(h) * p.D + lane * VEC), a);
        V::unpack(V::load(static_cast<const T*>(p.o) + row * p.o_stride + static_cast<long long>(h) * p.D + lane * VEC), b);
#pragma unroll
        for (int e = 0; e < VEC; ++e) s = fmaf(a[e], b[e], s);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (live && lane == 0) p.delta[static_cast<long long>(h) * p.q_rows + row] = s;
}

}  // namespace attn
}  // namespace eqlin
