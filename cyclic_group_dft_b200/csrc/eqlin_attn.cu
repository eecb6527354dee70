// eqlin_attn.cu -- host side of attention over packed sequences (include/eqlin.h): argument
// checks, the choice of kernels and their launches.
#include <algorithm>
#include <cmath>

#include <cudaTypedefs.h>

#include <mutex>

#include "eqlin_attn.cuh"
#include "eqlin_attn_f32.cuh"
#include "eqlin_attn_bwd_tc.cuh"
#include "eqlin_attn_mma.cuh"
#include "eqlin_attn_tc.cuh"
#include "eqlin_host_util.h"

namespace {

using namespace eqlin::host;
using eqlin::report;
namespace attn = eqlin::attn;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1024;   // rows past the end of the last tile are counted in 32 bits too
constexpr int64_t kMaxStride = int64_t(1) << 38;   // (a TMA stride is below 2^40 bytes)

int check_shape(const eqlin_attention_shape* a) {
    if (!a) return report(EQLIN_ERR_INVALID_ARG, "shape is NULL");
    if (a->q_rows < 0 || a->k_rows < 0 || a->heads < 1 || a->kv_heads < 1 || a->head_dim < 1 || a->sequences < 1)
        return report(EQLIN_ERR_INVALID_ARG, "row counts must be >= 0; heads, kv_heads, head_dim, sequences >= 1");
    if (!known_dtype(a->io_dtype)) return report(EQLIN_ERR_INVALID_ARG, "unknown dtype");
    if (a->heads % a->kv_heads) return report(EQLIN_ERR_INVALID_ARG, "heads must be a multiple of kv_heads");
    if (!(a->scale > 0.f) || !std::isfinite(a->scale))
        return report(EQLIN_ERR_INVALID_ARG, "scale must be finite and positive");
    if (a->causal != 0 && a->causal != 1) return report(EQLIN_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (!a->q_offsets != !a->k_offsets)
        return report(EQLIN_ERR_INVALID_ARG, "q_offsets and k_offsets go together");
    if (!a->q_offsets && a->sequences != 1)
        return report(EQLIN_ERR_INVALID_ARG, "several sequences need q_offsets and k_offsets");
    if (a->head_dim % 8 || a->head_dim > 128)
        return report(EQLIN_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 and at most 128");
    if (a->heads > 65535 || a->q_rows >= kMaxRows || a->k_rows >= kMaxRows || a->sequences >= (int64_t(1) << 24))
        return report(EQLIN_ERR_UNSUPPORTED, "fewer than 65536 heads, 2^31 - 1024 rows and 2^24 sequences are supported");
    if (!aligned(a->q_offsets, 4) || !aligned(a->k_offsets, 4))
        return report(EQLIN_ERR_MISALIGNED, "the offsets must be 4-byte aligned");
    return EQLIN_OK;
}

// One tensor of `rows` rows of `width` features: stride and address.
int check_tensor(const void* t, int64_t rows, int64_t width, int64_t stride, int io, const char* what) {
    if (rows == 0) return EQLIN_OK;
    if (!t) return report(EQLIN_ERR_INVALID_ARG, what);
    const int vec = 16 / elem_bytes(io);
    if (stride < width || stride > kMaxStride) return report(EQLIN_ERR_INVALID_ARG, "a row stride is smaller than its row, or too large");
    if (stride % vec || !aligned(t, 16))
        return report(EQLIN_ERR_MISALIGNED, "rows must be 16-byte aligned (address and stride)");
    return EQLIN_OK;
}

// fp32: blocks along x
unsigned slots(int64_t rows, int64_t sequences, int m) { return static_cast<unsigned>(rows / m + sequences); }

void fill(const eqlin_attention_shape* a, attn::Params& p) {
    p.q_offsets = a->q_offsets;
    p.k_offsets = a->k_offsets;
    p.q_stride = a->q_stride;
    p.k_stride = a->k_stride;
    p.v_stride = a->v_stride;
    p.o_stride = a->o_stride;
    p.q_rows = static_cast<int>(a->q_rows);
    p.k_rows = static_cast<int>(a->k_rows);
    p.sequences = static_cast<int>(a->sequences);
    p.heads = static_cast<int>(a->heads);
    p.kv_heads = static_cast<int>(a->kv_heads);
    p.D = static_cast<int>(a->head_dim);
    p.causal = a->causal;
    p.scale = a->scale;
}

// ---------------------------------------------------------------- tensor cores (16-bit I/O)
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// Tensor [rows][heads][D], rows `stride` features apart, read in boxes of 64 features of one head and
// box_rows rows with 128-byte swizzle.  Coordinates are (0 or 64, head, row): every copy starts on a
// 16-byte boundary.  What lies outside the tensor, features past D among it, reads as zero.
int encode_map(const void* t, int64_t rows, int64_t heads, int64_t D, int64_t stride, int io, CUtensorMap* map,
               int box_rows = attn::tc::kTile) {
    auto encode = tensor_map_encoder();
    if (!encode) return report(EQLIN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(D * 2), static_cast<cuuint64_t>(stride * 2)};
    cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = encode(map, io == EQLIN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                              const_cast<void*>(t), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? EQLIN_OK : report(EQLIN_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

// Grid of `heads` blocks for each slot, or an error where that is more than a launch takes.
int tc_grid(int64_t rows, int64_t sequences, int m, int64_t heads, unsigned* grid) {
    const int64_t n = (rows / m + sequences) * heads;
    if (n >= (int64_t(1) << 31)) return report(EQLIN_ERR_UNSUPPORTED, "too many rows, sequences and heads for one call");
    *grid = static_cast<unsigned>(n);
    return EQLIN_OK;
}

// The same for the kernels of short sequences.
template <int M>
int short_grid(int64_t rows, int64_t sequences, int64_t head_blocks, unsigned* grid, int64_t per = 1) {
    const int64_t n = attn::mma::short_blocks<M>(rows, sequences, per) * head_blocks;
    if (n >= (int64_t(1) << 31)) return report(EQLIN_ERR_UNSUPPORTED, "too many rows, sequences and heads for one call");
    *grid = static_cast<unsigned>(n);
    return EQLIN_OK;
}

// Limits of the bounded waits; EQLIN_WAIT_TIMEOUT_MS and the test hook EQLIN_TEST_STOP_AFTER (the load
// warp stops after that many tiles, so that the waits run out) are read on each call.
unsigned long long wait_timeout_ns() {
    const char* t = std::getenv("EQLIN_WAIT_TIMEOUT_MS");
    const long long ms = t ? std::atoll(t) : 0;
    return ms > 0 ? static_cast<unsigned long long>(ms) * 1000000ull : 2000000000ull;
}
long long stop_after() {
    const char* t = std::getenv("EQLIN_TEST_STOP_AFTER");
    return t ? std::atoll(t) : -1;
}

template <class T, int DP, int NQ>
int forward_tc(attn::tc::FwdParams fp, int io, cudaStream_t st) {
    using F = attn::tc::Fwd<DP, NQ>;
    attn::Params& p = fp.p;
    CUtensorMap mq, mk, mv;
    unsigned grid = 0;
    int s = tc_grid(p.q_rows, p.sequences, NQ * attn::tc::kTile, p.heads, &grid);
    if (s == EQLIN_OK) s = encode_map(p.q, p.q_rows, p.heads, p.D, p.q_stride, io, &mq);
    mk = mv = mq;   // without keys neither is read
    if (s == EQLIN_OK && p.k_rows > 0) s = encode_map(p.k, p.k_rows, p.kv_heads, p.D, p.k_stride, io, &mk);
    if (s == EQLIN_OK && p.k_rows > 0) s = encode_map(p.v, p.k_rows, p.kv_heads, p.D, p.v_stride, io, &mv);
    if (s != EQLIN_OK) return s;
    return launch(attn::tc::eqlin_attn_fwd_tc_kernel<T, DP, NQ>, dim3(grid), dim3(F::THREADS), F::SMEM, st,
                  "attention launch", mq, mk, mv, fp);
}
// ------------------------------------------------------------------------ choice of the forward
enum class Fwd { kTiles, kShort, kFew };

constexpr int kB200Sms = 148;   // the plans do not depend on the device, so that sizes need none

// By the average lengths, which the host knows (the single ones are device data); every kernel is right
// for every length.  Measured in bf16, us, 8 heads unless said otherwise.
//   few    tiles of 16 packed rows (queries times heads of a key head), keys split over the SMs.  Taken
//          - where its tiles do not fill the SMs and the keys can be split: 32 queries over 4096 keys, 8 sequences,
//            64 features: 21, tiles 39, short 83; 512 keys: 8.6, 11, 15;
//          - where packing reads the keys several times less often: 8 queries, 2 key heads, 512 keys, 64
//            sequences: 12.7, short 17, tiles 19; 2048 keys: 24, 54, 46.  Below 512 keys its join costs more: 128
//            keys, 256 sequences, 8 queries 29, short 19, but 1 query 15, 19;
//          - for up to 16 packed rows over long keys: 1 query, 2048 keys, 64 sequences, 128 features 95, short 95,
//            tiles 118.
//   short  tiles of 64 rows without a pipeline over the keys, several blocks to an SM.  Up to 64 rows on both sides
//          (49, 4096 sequences, 3 heads of 128 features: 143, tiles 539); with blocks enough also up to 128 (128,
//          1024 sequences, 3 heads of 128: 138, tiles 175; 192: 195, 177; but 16 sequences of 4 heads: 21, 6.6), or
//          512 keys for 64 queries (512 keys, 64 sequences, 64 queries: 25, tiles 27; 2048: 93, 68).
//   tiles  the rest: tcgen05.
Fwd forward_kind(const eqlin_attention_shape& a) {
    if (a.io_dtype == EQLIN_F32) return Fwd::kTiles;
    const int64_t n = a.sequences, packed = a.q_rows * (a.heads / a.kv_heads);
    const int64_t few_tiles = std::max(n, (packed + 15) / 16) * a.kv_heads;     // blocks without splits
    const int64_t short_tiles = std::max(n, (a.q_rows + 63) / 64) * a.heads;
    if (a.k_rows >= 128 * n && packed < kMaxRows) {   // (packed rows are counted in 32 bits)
        const bool longer = a.k_rows >= 512 * n;
        if (few_tiles <= kB200Sms && (packed <= 16 * n || (packed <= 128 * n && longer))) return Fwd::kFew;
        if (few_tiles * (longer ? 2 : 4) <= short_tiles) return Fwd::kFew;
        if (packed <= 16 * n && a.k_rows >= 1024 * n) return Fwd::kFew;
    }
    if (a.q_rows <= 64 * n && a.k_rows <= 64 * n) return Fwd::kShort;
    if (short_tiles >= 3 * kB200Sms &&
        ((a.q_rows <= 128 * n && a.k_rows <= 128 * n) || (a.q_rows <= 64 * n && a.k_rows <= 512 * n)))
        return Fwd::kShort;
    return Fwd::kTiles;
}

// fp32: 16-row tiles on the CUDA cores, with split keys in the forward, where few tiles of 64 rows would be left
// for the tensor cores.  Measured, 64 features, CUDA cores / tensor cores: 16 tiles (256 tokens, 4 heads) forward
// 17 / 21 us, gradients 41 / 64; 32 tiles 31 / 37 and 89 / 117; 48 tiles 27 / 21 and 68 / 66; 64 tiles (1024
// tokens, 4 heads) 91 / 70 and 290 / 232.
int64_t f32_tiles(int64_t rows, int64_t sequences, int64_t heads) {
    return std::max(sequences, (rows + 63) / 64) * heads;
}
bool f32_small(int64_t rows, int64_t sequences, int64_t heads) {
    return f32_tiles(rows, sequences, heads) < kB200Sms / 4;
}
// Forward: few queries too, as long as splits help (1 query over 4096 keys, 8 heads, 16 sequences: 179 / 285 us;
// 16 queries, 32 sequences: 344 / 294).
bool f32_small_forward(int64_t rows, int64_t sequences, int64_t heads) {
    return f32_tiles(rows, sequences, heads) < (rows <= 16 * sequences ? kB200Sms : kB200Sms / 4);
}

// Slices of the keys, where the tiles alone would leave SMs idle: as many as fill them once, but no slice below 256
// keys.  fp32: tiles of 16 rows, two blocks to an SM for heads of up to 64 features.  Above, one fits, and twice as many
// slices run in two waves, which costs as often as it gains, for 148 blocks / 296: 128 features, 48 queries, 2048 keys, 8
// heads 42 / 53 us; 1 query, 4096 keys, 4 sequences, 8 heads 99 / 96; 64 queries, 8192 keys, 8 heads 190 / 182; 100
// queries, 1500 keys, 2 sequences, 4 heads 74 / 65.
int forward_splits(const eqlin_attention_shape& a) {
    const Fwd kind = forward_kind(a);
    const int64_t keys = a.k_rows / a.sequences;
    int64_t units, room;
    if (kind == Fwd::kFew) {
        const int64_t rows = a.q_rows * (a.heads / a.kv_heads);
        units = std::max(a.sequences, (rows + 15) / 16) * a.kv_heads;
        room = kB200Sms;
    } else if (a.io_dtype == EQLIN_F32 && f32_small_forward(a.q_rows, a.sequences, a.heads)) {
        units = std::max(a.sequences, (a.q_rows + 15) / 16) * a.heads;
        room = 2 * kB200Sms;
    } else {
        return 1;
    }
    return static_cast<int>(std::max<int64_t>(1, std::min({room / std::max<int64_t>(units, 1), keys / 256, int64_t(64)})));
}

// 16-bit gradients by 16-row products: up to 64 rows on both sides (49, 4096 sequences, 3 heads of 128 features: 326
// us, tcgen05 tiles 1241; 96: 846, 796).  With blocks enough, also few queries over more keys, which leave the tiles of
// 128 empty: up to 64 over 128 keys (64 queries, 256 sequences, 8 heads of 64: 107 us, tiles 136), and up to
// 32 where key heads are not shared (1 query, 2048 keys, 64 sequences, 8 heads of 64: 230, 280; of 2 key heads:
// 177, 146; 8 sequences of 4096 keys: 171, 101).
bool backward_short_rows(int64_t q_rows, int64_t k_rows, int64_t n, int64_t heads, int64_t kv_heads) {
    if (std::max(q_rows, k_rows) <= 64 * n) return true;
    return n * heads >= 3 * kB200Sms && q_rows <= 64 * n &&
           (k_rows <= 128 * n || (heads == kv_heads && q_rows <= 32 * n));
}

size_t backward_workspace(const eqlin_attention_shape& a) {
    if (a.io_dtype == EQLIN_F32 || backward_short_rows(a.q_rows, a.k_rows, a.sequences, a.heads, a.kv_heads))
        return size_t(a.q_rows) * size_t(a.heads) * sizeof(float);
    const size_t q_tiles = size_t(a.q_rows / attn::tc::kTile + a.sequences) * size_t(a.heads);
    const size_t k_tiles = size_t(a.k_rows / attn::tc::kTile + a.sequences) * size_t(a.kv_heads);
    const size_t floats = q_tiles * 2 * attn::tc::kTile;     // lse and delta
    return (a.io_dtype == EQLIN_F16 ? floats + q_tiles * 16 + k_tiles * 4 : floats) * sizeof(float);
}

size_t forward_workspace(const eqlin_attention_shape& a) {
    const int n = forward_splits(a);
    return n == 1 ? 0 : size_t(n) * size_t(a.heads) * size_t(a.q_rows) * size_t(a.head_dim + 1) * sizeof(float);
}

template <class T>
int launch_join(const attn::Params& p, cudaStream_t st) {
    const long long units = static_cast<long long>(p.q_rows) * p.heads;
    return launch(attn::eqlin_attn_join_kernel<T>, dim3(static_cast<unsigned>((units + 3) / 4)), dim3(128), 0, st,
                  "attention launch", p);
}

template <class T, int DP, int M>
int forward_short_m(const attn::Params& p, cudaStream_t st) {
    constexpr int U = 64 / M;
    unsigned grid = 0;
    const int s = short_grid<M>(p.q_rows, p.sequences, (p.heads + U - 1) / U, &grid);
    if (s != EQLIN_OK) return s;
    return launch(attn::mma::eqlin_attn_fwd_short_kernel<T, DP, M>, dim3(grid), dim3(attn::mma::kShortThreads),
                  attn::mma::short_smem<T, DP>(), st, "attention launch", p);
}
template <class T, int DP>
int forward_short(const attn::Params& p, cudaStream_t st) {
    const int64_t rows = std::max(p.q_rows, p.k_rows);
    if (rows <= int64_t(16) * p.sequences) return forward_short_m<T, DP, 16>(p, st);
    if (rows <= int64_t(32) * p.sequences) return forward_short_m<T, DP, 32>(p, st);
    return forward_short_m<T, DP, 64>(p, st);
}

template <class T, int DP>
int forward_few(const attn::Params& p, cudaStream_t st) {
    using F = attn::mma::Few<DP>;
    const int64_t rows = int64_t(p.q_rows) * (p.heads / p.kv_heads);
    unsigned grid = 0;
    int s = tc_grid(rows, p.sequences, 16, int64_t(p.kv_heads) * p.splits, &grid);
    if (s != EQLIN_OK) return s;
    s = launch(attn::mma::eqlin_attn_fwd_few_kernel<T, DP>, dim3(grid), dim3(F::WARPS * 32), F::SMEM, st,
               "attention launch", p);
    return s == EQLIN_OK && p.splits > 1 ? launch_join<T>(p, st) : s;
}

template <class T>
int forward_16(attn::Params& p, Fwd kind, int io, cudaStream_t st) {
    if (kind == Fwd::kShort) return p.D <= 64 ? forward_short<T, 64>(p, st) : forward_short<T, 128>(p, st);
    if (kind == Fwd::kFew) return p.D <= 64 ? forward_few<T, 64>(p, st) : forward_few<T, 128>(p, st);
    p.timeout_ns = wait_timeout_ns();
    attn::tc::FwdParams fp = {p, stop_after()};
    return p.D <= 64 ? forward_tc<T, 64, 1>(fp, io, st) : forward_tc<T, 128, 2>(fp, io, st);
}

// ------------------------------------------------------------------------------------ fp32 I/O
template <int DP>
int forward_f32_small(const attn::Params& p, cudaStream_t st) {
    using namespace attn::f32;
    using S = Shape<DP>;
    const int s = launch(eqlin_attn_fwd_f32_kernel<DP>, dim3(slots(p.q_rows, p.sequences, S::M), p.heads, p.splits),
                         dim3(kThreads), S::FWD_BYTES, st, "attention launch", p);
    return s == EQLIN_OK && p.splits > 1 ? launch_join<float>(p, st) : s;
}
template <int DP>
int forward_f32_tiles(const attn::Params& p, cudaStream_t st) {
    unsigned grid = 0;
    const int s = tc_grid(p.q_rows, p.sequences, 64, p.heads, &grid);
    if (s != EQLIN_OK) return s;
    return launch(attn::mma::eqlin_attn_fwd_f32_kernel<DP>, dim3(grid), dim3(attn::mma::kShortThreads),
                  attn::mma::short_smem<float, DP>(), st, "attention launch", p);
}
int forward_f32(const attn::Params& p, cudaStream_t st) {
    if (f32_small_forward(p.q_rows, p.sequences, p.heads))
        return p.D <= 64 ? forward_f32_small<64>(p, st) : forward_f32_small<128>(p, st);
    return p.D <= 64 ? forward_f32_tiles<64>(p, st) : forward_f32_tiles<128>(p, st);
}

template <class T>
int launch_delta(const attn::Params& p, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    int lanes = 1;
    while (lanes * VEC < p.D) lanes *= 2;
    const long long units = static_cast<long long>(p.q_rows) * p.heads;
    const long long blocks = (units + 256 / lanes - 1) / (256 / lanes);
    return launch(attn::eqlin_attn_delta_kernel<T, VEC>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st,
                  "attention gradient launch", p, lanes);
}

template <int DP>
int backward_f32_small(const attn::Params& p, cudaStream_t st) {
    using namespace attn::f32;
    using S = Shape<DP>;
    unsigned k_blocks = 0, q_blocks = 0;
    int s = EQLIN_OK;
    if (p.k_rows > 0) s = tc_grid(p.k_rows, p.sequences, S::M, p.kv_heads, &k_blocks);
    if (s == EQLIN_OK && p.q_rows > 0) s = tc_grid(p.q_rows, p.sequences, S::M, p.heads, &q_blocks);
    if (s == EQLIN_OK && int64_t(k_blocks) + q_blocks >= (int64_t(1) << 31))
        s = report(EQLIN_ERR_UNSUPPORTED, "too many rows, sequences and heads for one call");
    if (s == EQLIN_OK && p.q_rows > 0) s = launch_delta<float>(p, st);
    if (s != EQLIN_OK) return s;
    return launch(eqlin_attn_bwd_f32_kernel<DP>, dim3(k_blocks + q_blocks), dim3(kThreads),
                  std::max(S::DKV_BYTES, S::DQ_BYTES), st, "attention gradient launch", p, k_blocks);
}
template <int DP>
int backward_f32_tiles(const attn::Params& p, cudaStream_t st) {
    namespace mma = attn::mma;
    unsigned grid_q = 0, grid_k = 0;
    int s = tc_grid(p.q_rows, p.sequences, 64, p.heads, &grid_q);
    if (s == EQLIN_OK) s = tc_grid(p.k_rows, p.sequences, 64, p.kv_heads, &grid_k);
    if (s == EQLIN_OK && p.q_rows > 0)
        s = launch(mma::eqlin_attn_dq_f32_kernel<DP>, dim3(grid_q), dim3(mma::kShortThreads),
                   mma::short_bwd_smem<float, DP>(), st, "attention gradient launch", p);
    if (s == EQLIN_OK && p.k_rows > 0)
        s = launch(mma::eqlin_attn_dkv_f32_kernel<DP>, dim3(grid_k), dim3(mma::kShortThreads),
                   mma::short_bwd_smem<float, DP>(), st, "attention gradient launch", p);
    return s;
}
int backward_f32(const attn::Params& p, cudaStream_t st) {
    if (f32_small(std::max(p.q_rows, p.k_rows), p.sequences, p.heads))
        return p.D <= 64 ? backward_f32_small<64>(p, st) : backward_f32_small<128>(p, st);
    return p.D <= 64 ? backward_f32_tiles<64>(p, st) : backward_f32_tiles<128>(p, st);
}

template <class T, int DP>
int backward_tc(attn::tc::BwdParams bp, int io, cudaStream_t st) {
    namespace tc = attn::tc;
    using B = tc::Bwd<DP>;
    attn::Params& p = bp.p;
    unsigned grid_k = 0, grid_q = 0;
    int s = tc_grid(p.k_rows, p.sequences, tc::kTile, p.kv_heads, &grid_k);
    if (s == EQLIN_OK) s = tc_grid(p.q_rows, p.sequences, tc::kTile, p.heads, &grid_q);
    CUtensorMap mq, mk, mv, mdo;
    if (s == EQLIN_OK && p.q_rows > 0) {
        s = encode_map(p.q, p.q_rows, p.heads, p.D, p.q_stride, io, &mq, B::LOAD_ROWS);
        if (s == EQLIN_OK) s = encode_map(p.dout, p.q_rows, p.heads, p.D, p.do_stride, io, &mdo, B::LOAD_ROWS);
    }
    if (s == EQLIN_OK && p.k_rows > 0) {
        s = encode_map(p.k, p.k_rows, p.kv_heads, p.D, p.k_stride, io, &mk, B::LOAD_ROWS);
        if (s == EQLIN_OK) s = encode_map(p.v, p.k_rows, p.kv_heads, p.D, p.v_stride, io, &mv, B::LOAD_ROWS);
    }
    if (s != EQLIN_OK) return s;
    if (p.q_rows == 0) mq = mdo = mk;   // the side without rows is never read
    if (p.k_rows == 0) mk = mv = mq;
    p.do_most = p.delta + size_t(grid_q) * 2 * tc::kTile;   // in the order of backward_workspace
    p.v_most = p.do_most + size_t(grid_q) * 16;
    if (p.q_rows > 0)
        s = launch(tc::eqlin_attn_stats_kernel<T>, dim3(grid_q), dim3(256), 0, st, "attention gradient launch", p);
    if (s == EQLIN_OK && p.k_rows > 0)
        s = launch(tc::eqlin_attn_dkv_tc_kernel<T, DP>, dim3(grid_k), dim3(B::THREADS), B::SMEM, st,
                   "attention gradient launch", mq, mk, mv, mdo, bp);
    if (s == EQLIN_OK && p.q_rows > 0)
        s = launch(tc::eqlin_attn_dq_tc_kernel<T, DP>, dim3(grid_q), dim3(B::THREADS), B::SMEM, st,
                   "attention gradient launch", mq, mk, mv, mdo, bp);
    return s;
}
template <class T, int DP, int M>
int backward_short_m(const attn::Params& p, cudaStream_t st) {
    namespace mma = attn::mma;
    constexpr int U = 64 / M;
    unsigned grid_q = 0, grid_k = 0;
    int s = short_grid<M>(p.q_rows, p.sequences, (p.heads + U - 1) / U, &grid_q);
    // sequences to a block of the second launch, which skips those of one tile: as many as leave the SMs several
    // blocks each
    const int64_t hb = (p.kv_heads + U - 1) / U;
    const int per = p.heads != p.kv_heads ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(32, p.sequences * hb / (4 * kB200Sms))));
    if (s == EQLIN_OK) s = short_grid<M>(p.k_rows, p.sequences, hb, &grid_k, per);
    if (s == EQLIN_OK && p.q_rows > 0)
        s = launch(mma::eqlin_attn_dq_short_kernel<T, DP, M>, dim3(grid_q), dim3(mma::kShortThreads),
                   mma::short_bwd_smem<T, DP>(), st, "attention gradient launch", p);
    if (s == EQLIN_OK && p.k_rows > 0)
        s = launch(mma::eqlin_attn_dkv_short_kernel<T, DP, M>, dim3(grid_k), dim3(mma::kShortThreads),
                   mma::short_bwd_smem<T, DP>(), st, "attention gradient launch", p, per);
    return s;
}
template <class T, int DP>
int backward_short(const attn::Params& p, cudaStream_t st) {
    const int64_t rows = std::max(p.q_rows, p.k_rows);
    if (rows <= int64_t(16) * p.sequences) return backward_short_m<T, DP, 16>(p, st);
    if (rows <= int64_t(32) * p.sequences) return backward_short_m<T, DP, 32>(p, st);
    return backward_short_m<T, DP, 64>(p, st);
}

template <class T>
int backward_16(attn::Params& p, int io, cudaStream_t st) {
    if (backward_short_rows(p.q_rows, p.k_rows, p.sequences, p.heads, p.kv_heads))
        return p.D <= 64 ? backward_short<T, 64>(p, st) : backward_short<T, 128>(p, st);
    p.timeout_ns = wait_timeout_ns();
    const attn::tc::BwdParams bp = {p, stop_after()};
    return p.D <= 64 ? backward_tc<T, 64>(bp, io, st) : backward_tc<T, 128>(bp, io, st);
}

}  // namespace

extern "C" {

int eqlin_attention_workspace_size(const eqlin_attention_shape* shape, int backward, size_t* bytes) {
    if (!bytes) return report(EQLIN_ERR_INVALID_ARG, "NULL argument");
    const int s = check_shape(shape);
    if (s != EQLIN_OK) return s;
    *bytes = backward ? backward_workspace(*shape) : forward_workspace(*shape);
    return EQLIN_OK;
}

int eqlin_attention_forward(const eqlin_attention_shape* shape, const void* q, const void* k, const void* v, void* o,
                            float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    int s = check_shape(shape);
    if (s != EQLIN_OK) return s;
    const eqlin_attention_shape& a = *shape;
    const int64_t wq = a.heads * a.head_dim, wk = a.kv_heads * a.head_dim;
    if ((s = check_tensor(q, a.q_rows, wq, a.q_stride, a.io_dtype, "q is NULL")) != EQLIN_OK ||
        (s = check_tensor(k, a.k_rows, wk, a.k_stride, a.io_dtype, "k is NULL")) != EQLIN_OK ||
        (s = check_tensor(v, a.k_rows, wk, a.v_stride, a.io_dtype, "v is NULL")) != EQLIN_OK ||
        (s = check_tensor(o, a.q_rows, wq, a.o_stride, a.io_dtype, "o is NULL")) != EQLIN_OK)
        return s;
    if (!aligned(lse, 4)) return report(EQLIN_ERR_MISALIGNED, "lse must be 4-byte aligned");
    size_t need = 0;
    if ((s = eqlin_attention_workspace_size(shape, 0, &need)) != EQLIN_OK) return s;
    if (need && (!workspace || workspace_bytes < need))
        return report(EQLIN_ERR_INVALID_ARG, "workspace missing or smaller than eqlin_attention_workspace_size");
    if (!aligned(workspace, 16)) return report(EQLIN_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    if (a.q_rows == 0) return EQLIN_OK;
    int sms = 0;
    if ((s = current_device(nullptr, &sms)) != EQLIN_OK) return s;
    attn::Params p = {};
    fill(shape, p);
    p.q = q;
    p.k = k;
    p.v = v;
    p.out = o;
    p.lse = lse;
    p.splits = forward_splits(a);
    p.part_o = static_cast<float*>(workspace);
    if (p.splits > 1) p.part_lse = p.part_o + size_t(p.splits) * a.heads * a.q_rows * a.head_dim;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a.io_dtype == EQLIN_F32) return forward_f32(p, st);
    const Fwd kind = forward_kind(a);
    return a.io_dtype == EQLIN_F16 ? forward_16<__half>(p, kind, a.io_dtype, st)
                                   : forward_16<__nv_bfloat16>(p, kind, a.io_dtype, st);
}

int eqlin_attention_device_status(int* status_out) {
    if (!status_out) return report(EQLIN_ERR_INVALID_ARG, "NULL argument");
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return eqlin::report_cuda(e, "cudaDeviceSynchronize");
    int v = 0;
    const int zero = 0;
    if ((e = cudaMemcpyFromSymbol(&v, attn::g_status, sizeof(v))) != cudaSuccess ||
        (e = cudaMemcpyToSymbol(attn::g_status, &zero, sizeof(zero))) != cudaSuccess)
        return eqlin::report_cuda(e, "status read");
    *status_out = v;
    return EQLIN_OK;
}

int eqlin_attention_backward(const eqlin_attention_shape* shape, const eqlin_attention_grad_strides* strides,
                             const void* dout, const void* q, const void* k, const void* v, const void* o,
                             const float* lse, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                             void* stream) {
    int s = check_shape(shape);
    if (s != EQLIN_OK) return s;
    if (!strides) return report(EQLIN_ERR_INVALID_ARG, "strides is NULL");
    const eqlin_attention_shape& a = *shape;
    const int64_t wq = a.heads * a.head_dim, wk = a.kv_heads * a.head_dim;
    const int io = a.io_dtype;
    if ((s = check_tensor(q, a.q_rows, wq, a.q_stride, io, "q is NULL")) != EQLIN_OK ||
        (s = check_tensor(k, a.k_rows, wk, a.k_stride, io, "k is NULL")) != EQLIN_OK ||
        (s = check_tensor(v, a.k_rows, wk, a.v_stride, io, "v is NULL")) != EQLIN_OK ||
        (s = check_tensor(o, a.q_rows, wq, a.o_stride, io, "o is NULL")) != EQLIN_OK ||
        (s = check_tensor(dout, a.q_rows, wq, strides->dout, io, "dout is NULL")) != EQLIN_OK ||
        (s = check_tensor(dq, a.q_rows, wq, strides->dq, io, "dq is NULL")) != EQLIN_OK ||
        (s = check_tensor(dk, a.k_rows, wk, strides->dk, io, "dk is NULL")) != EQLIN_OK ||
        (s = check_tensor(dv, a.k_rows, wk, strides->dv, io, "dv is NULL")) != EQLIN_OK)
        return s;
    if (a.q_rows > 0 && !lse) return report(EQLIN_ERR_INVALID_ARG, "lse is NULL");
    if (!aligned(lse, 4)) return report(EQLIN_ERR_MISALIGNED, "lse must be 4-byte aligned");
    size_t need = 0;
    if ((s = eqlin_attention_workspace_size(shape, 1, &need)) != EQLIN_OK) return s;
    if (need && (!workspace || workspace_bytes < need))
        return report(EQLIN_ERR_INVALID_ARG, "workspace missing or smaller than eqlin_attention_workspace_size");
    if (!aligned(workspace, 16)) return report(EQLIN_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    if (a.q_rows == 0 && a.k_rows == 0) return EQLIN_OK;
    int sms = 0;
    if ((s = current_device(nullptr, &sms)) != EQLIN_OK) return s;
    attn::Params p = {};
    fill(shape, p);
    p.q = q;
    p.k = k;
    p.v = v;
    p.o = o;
    p.dout = dout;
    p.lse = const_cast<float*>(lse);
    p.delta = static_cast<float*>(workspace);
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.do_stride = strides->dout;
    p.dq_stride = strides->dq;
    p.dk_stride = strides->dk;
    p.dv_stride = strides->dv;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (io == EQLIN_F32) return backward_f32(p, st);
    return io == EQLIN_F16 ? backward_16<__half>(p, io, st) : backward_16<__nv_bfloat16>(p, io, st);
}

}  // extern "C"
