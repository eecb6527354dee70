// eqlin_block.cu -- host side of the memory-bound operators around the layers (include/eqlin.h):
// residual addition with root-mean-square norm, its 8-bit form and its gradients, and rotary
// positions.
#include <algorithm>
#include <cmath>

#include "eqlin_host_util.h"
#include "eqlin_norm.cuh"
#include "eqlin_rope.cuh"

namespace {

using namespace eqlin::host;
using eqlin::report;
namespace norm = eqlin::norm;
namespace rope = eqlin::rope;

// ------------------------------------------------------------------------- norm
struct NormPlan {
    int vec = 0, vpt = 0, tpr = 0;
    bool wide = false;
    unsigned blocks = 0;
};

// Threads of a row and vectors of a thread: among 1..4 vectors and powers of two of threads,
// the pair that covers the row with the fewest idle vectors; among equals the one with more
// vectors per thread (fewer shuffle steps, more loads in flight).  p4 C = 96 in 16 bits: 48
// vectors, 16 threads of 3.
int plan_norm(int64_t N, int64_t C, int64_t G, int io, int sms, bool backward, NormPlan* pl) {
    const int64_t L = C * G;
    const int full = io == EQLIN_F32 ? 4 : 8;
    pl->vec = L % full == 0 ? full : 1;
    const int64_t nv = L / pl->vec;
    int64_t best = -1;
    for (int vpt = 1; vpt <= norm::kMaxVpt; ++vpt) {
        int tpr = 1;
        while (int64_t(tpr) * vpt < nv && tpr < norm::kMaxWide) tpr *= 2;
        if (int64_t(tpr) * vpt < nv) continue;
        if (best < 0 || int64_t(tpr) * vpt <= best) {
            best = int64_t(tpr) * vpt;
            pl->vpt = vpt;
            pl->tpr = tpr;
        }
    }
    if (best < 0)
        return report(EQLIN_ERR_UNSUPPORTED, "C * G is too large for the norm (16384 features in 16 bits, 8192 in "
                                             "fp32, 2048 in fp32 when not a multiple of 4)");
    pl->wide = pl->tpr > 32;
    const int64_t groups = pl->wide ? 1 : norm::kThreads / pl->tpr;
    const int64_t rows = (N + groups - 1) / groups;
    const int fit = pl->wide ? norm::kMaxWide / pl->tpr : 1;   // the wide form's counts are for its largest block
    const int per_sm = fit * (backward ? norm::bwd_blocks(pl->vpt, pl->wide) : norm::fwd_blocks(pl->vpt, pl->wide));
    pl->blocks = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(rows, int64_t(sms) * per_sm)));
    return EQLIN_OK;
}

int check_norm(int64_t N, int64_t C, int64_t G, float eps, int w_dtype, int io, int* lg) {
    if (N < 0 || C < 1) return report(EQLIN_ERR_INVALID_ARG, "N must be >= 0 and C >= 1");
    if (!known_dtype(io) || !known_dtype(w_dtype)) return report(EQLIN_ERR_INVALID_ARG, "unknown dtype");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return report(EQLIN_ERR_INVALID_ARG, "eps must be finite and >= 0");
    *lg = log2_group(G);
    if (*lg < 0) return report(EQLIN_ERR_UNSUPPORTED, "G must be 1, 2, 4, 8 or 16");
    if (N >= (int64_t(1) << 31)) return report(EQLIN_ERR_UNSUPPORTED, "N must be below 2^31");
    if (C > (int64_t(1) << 16)) return report(EQLIN_ERR_UNSUPPORTED, "C must be at most 65536");
    if (io != EQLIN_F32 && (C * G) % 8 != 0)
        return report(EQLIN_ERR_UNSUPPORTED, "16-bit I/O needs C * G to be a multiple of 8 (16-byte rows)");
    return EQLIN_OK;
}

// Calls f(kernel tag) for the plan's instance.
template <class T, int VEC, class F>
int with_vpt(const NormPlan& pl, F&& f) {
    switch (pl.vpt * 2 + (pl.wide ? 1 : 0)) {
        case 2: return f(std::integral_constant<int, 1>(), std::false_type());
        case 3: return f(std::integral_constant<int, 1>(), std::true_type());
        case 4: return f(std::integral_constant<int, 2>(), std::false_type());
        case 5: return f(std::integral_constant<int, 2>(), std::true_type());
        case 6: return f(std::integral_constant<int, 3>(), std::false_type());
        case 7: return f(std::integral_constant<int, 3>(), std::true_type());
        case 8: return f(std::integral_constant<int, 4>(), std::false_type());
        default: return f(std::integral_constant<int, 4>(), std::true_type());
    }
}

template <class T, int VEC, bool OUT8>
int launch_norm_fwd(const NormPlan& pl, const norm::Params& p, cudaStream_t st) {
    return with_vpt<T, VEC>(pl, [&](auto vpt, auto wide) {
        return launch(norm::eqlin_add_rmsnorm_kernel<T, VEC, decltype(vpt)::value, decltype(wide)::value, OUT8>,
                      dim3(pl.blocks), dim3(pl.wide ? pl.tpr : norm::kThreads), 0, st, "norm launch", p);
    });
}

size_t bwd_smem(const NormPlan& pl, bool ring) {
    const int groups = pl.wide ? 1 : norm::kThreads / pl.tpr;
    const size_t weights = size_t(pl.tpr) * pl.vpt * pl.vec * sizeof(float), sums = groups * weights;
    return weights + std::max(sums, ring ? size_t(2) * 2 * pl.vpt * norm::kThreads * 16 : 0);
}

template <class T, int VEC>
int launch_norm_bwd(const NormPlan& pl, const norm::Params& p, cudaStream_t st) {
    return with_vpt<T, VEC>(pl, [&](auto vpt, auto wide) {
        constexpr int VPT = decltype(vpt)::value;
        constexpr bool WIDE = decltype(wide)::value, CAN = !WIDE && VEC * sizeof(T) == 16;
        auto go = [&](auto ring) {
            constexpr bool RING = decltype(ring)::value;
            return launch(norm::eqlin_rmsnorm_bwd_kernel<T, VEC, VPT, WIDE, RING>, dim3(pl.blocks),
                          dim3(pl.wide ? pl.tpr : norm::kThreads), bwd_smem(pl, RING), st, "norm gradient launch", p);
        };
        return CAN && !p.sum ? go(std::bool_constant<CAN>()) : go(std::false_type());
    });
}

int norm_forward(const void* x, const void* residual, const void* weight, void* y, float* scale, void* sum_out,
                 int64_t N, int64_t C, int64_t G, float eps, int w_dtype, int io, bool out8, void* stream) {
    int lg = 0;
    int s = check_norm(N, C, G, eps, w_dtype, io, &lg);
    if (s != EQLIN_OK) return s;
    NormPlan pl;
    if ((s = plan_norm(N, C, G, io, 1, false, &pl)) != EQLIN_OK) return s;   // sizes first, without a device
    if (N == 0) return EQLIN_OK;
    if (!x || !y || (out8 && !scale)) return report(EQLIN_ERR_INVALID_ARG, "x, y or scale is NULL");
    if (y == sum_out) return report(EQLIN_ERR_INVALID_ARG, "y and sum_out are the same tensor");
    if (out8 && (y == x || y == residual))   // rows of other sizes: one row's output lies over another's input
        return report(EQLIN_ERR_INVALID_ARG, "the 8-bit output cannot be written over its input");
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(sum_out, 16) || !aligned(scale, 4) ||
        !aligned(weight, elem_bytes(w_dtype)))
        return report(EQLIN_ERR_MISALIGNED, "x, residual, y and sum_out must be 16-byte aligned");
    int sms = 0;
    if ((s = current_device(nullptr, &sms)) != EQLIN_OK) return s;
    plan_norm(N, C, G, io, sms, false, &pl);
    norm::Params p = {};
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.y = y;
    p.sum = sum_out;
    p.scale = scale;
    p.N = N;
    p.L = static_cast<int>(C * G);
    p.C = static_cast<int>(C);
    p.lg_g = lg;
    p.tpr = pl.tpr;
    p.w_dtype = w_dtype;
    p.eps = eps;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (io == EQLIN_F32) {
        if (pl.vec == 4) return out8 ? launch_norm_fwd<float, 4, true>(pl, p, st) : launch_norm_fwd<float, 4, false>(pl, p, st);
        return out8 ? launch_norm_fwd<float, 1, true>(pl, p, st) : launch_norm_fwd<float, 1, false>(pl, p, st);
    }
    if (io == EQLIN_F16)
        return out8 ? launch_norm_fwd<__half, 8, true>(pl, p, st) : launch_norm_fwd<__half, 8, false>(pl, p, st);
    return out8 ? launch_norm_fwd<__nv_bfloat16, 8, true>(pl, p, st)
                : launch_norm_fwd<__nv_bfloat16, 8, false>(pl, p, st);
}

// ------------------------------------------------------------------------- rope
template <class T, int VEC>
int launch_rope(const rope::Params& p, unsigned blocks, size_t smem, cudaStream_t st) {
    return launch(rope::eqlin_rope_kernel<T, VEC>, dim3(blocks), dim3(rope::kThreads), smem, st, "rope launch", p);
}
template <class T>
int launch_rope_vec(int vec, const rope::Params& p, unsigned blocks, size_t smem, cudaStream_t st) {
    if constexpr (sizeof(T) == 2) {
        if (vec == 8) return launch_rope<T, 8>(p, blocks, smem, st);
    }
    if (vec == 4) return launch_rope<T, 4>(p, blocks, smem, st);
    if (vec == 2) return launch_rope<T, 2>(p, blocks, smem, st);
    return launch_rope<T, 1>(p, blocks, smem, st);
}

}  // namespace

extern "C" {

int eqlin_add_rmsnorm(const void* x, const void* residual, const void* weight, void* y, void* sum_out, int64_t N,
                      int64_t C, int64_t G, float eps, int w_dtype, int io_dtype, void* stream) {
    return norm_forward(x, residual, weight, y, nullptr, sum_out, N, C, G, eps, w_dtype, io_dtype, false, stream);
}

int eqlin_add_rmsnorm_fp8(const void* x, const void* residual, const void* weight, void* y8, float* scale,
                          void* sum_out, int64_t N, int64_t C, int64_t G, float eps, int w_dtype, int io_dtype,
                          void* stream) {
    return norm_forward(x, residual, weight, y8, scale, sum_out, N, C, G, eps, w_dtype, io_dtype, true, stream);
}

int eqlin_rmsnorm_backward_workspace_size(int64_t N, int64_t C, int64_t G, int io_dtype, size_t* bytes) {
    if (!bytes) return report(EQLIN_ERR_INVALID_ARG, "NULL argument");
    int lg = 0;
    int s = check_norm(N, C, G, 0.f, EQLIN_F32, io_dtype, &lg);
    if (s != EQLIN_OK) return s;
    NormPlan pl;
    // the most blocks that any sm_100 device of up to 256 SMs takes, so that no device is needed
    if ((s = plan_norm(N, C, G, io_dtype, 256, true, &pl)) != EQLIN_OK) return s;
    *bytes = N == 0 ? 0 : size_t(pl.blocks) * size_t(C) * sizeof(float);
    return EQLIN_OK;
}

int eqlin_rmsnorm_backward(const void* dy, const void* sum, const void* weight, const void* dsum, void* dx,
                           float* dweight, int64_t N, int64_t C, int64_t G, float eps, int w_dtype, int io_dtype,
                           void* workspace, size_t workspace_bytes, void* stream) {
    int lg = 0;
    int s = check_norm(N, C, G, eps, w_dtype, io_dtype, &lg);
    if (s != EQLIN_OK) return s;
    NormPlan pl;
    if ((s = plan_norm(N, C, G, io_dtype, 1, true, &pl)) != EQLIN_OK) return s;
    if (!aligned(dweight, 4)) return report(EQLIN_ERR_MISALIGNED, "dweight must be 4-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0) {   // the gradient of an empty batch is zero
        if (!dweight) return EQLIN_OK;
        const cudaError_t e = cudaMemsetAsync(dweight, 0, size_t(C) * sizeof(float), st);
        return e == cudaSuccess ? EQLIN_OK : eqlin::report_cuda(e, "dweight clear");
    }
    if (!dy || !sum || !dx) return report(EQLIN_ERR_INVALID_ARG, "dy, sum or dx is NULL");
    if (!aligned(dy, 16) || !aligned(sum, 16) || !aligned(dsum, 16) || !aligned(dx, 16) ||
        !aligned(weight, elem_bytes(w_dtype)))
        return report(EQLIN_ERR_MISALIGNED, "dy, sum, dsum and dx must be 16-byte aligned");
    if (dweight) {
        size_t need = 0;
        if ((s = eqlin_rmsnorm_backward_workspace_size(N, C, G, io_dtype, &need)) != EQLIN_OK) return s;
        if (!workspace || workspace_bytes < need)
            return report(EQLIN_ERR_INVALID_ARG,
                          "workspace missing or smaller than eqlin_rmsnorm_backward_workspace_size");
        if (!aligned(workspace, 16)) return report(EQLIN_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    }
    int sms = 0;
    if ((s = current_device(nullptr, &sms)) != EQLIN_OK) return s;
    plan_norm(N, C, G, io_dtype, std::min(sms, 256), true, &pl);
    norm::Params p = {};
    p.x = dy;
    p.residual = sum;
    p.weight = weight;
    p.y = dx;
    p.sum = const_cast<void*>(dsum);
    p.partial = dweight ? static_cast<float*>(workspace) : nullptr;
    p.N = N;
    p.L = static_cast<int>(C * G);
    p.C = static_cast<int>(C);
    p.lg_g = lg;
    p.tpr = pl.tpr;
    p.w_dtype = w_dtype;
    p.eps = eps;
    if (io_dtype == EQLIN_F32)
        s = pl.vec == 4 ? launch_norm_bwd<float, 4>(pl, p, st) : launch_norm_bwd<float, 1>(pl, p, st);
    else if (io_dtype == EQLIN_F16)
        s = launch_norm_bwd<__half, 8>(pl, p, st);
    else
        s = launch_norm_bwd<__nv_bfloat16, 8>(pl, p, st);
    if (s != EQLIN_OK || !dweight) return s;
    return launch(norm::eqlin_rmsnorm_dw_kernel, dim3(static_cast<unsigned>((C + 31) / 32)), dim3(32, 16), 0, st,
                  "norm weight gradient launch", static_cast<const float*>(p.partial), dweight, p.C,
                  static_cast<int>(pl.blocks));
}

int eqlin_rope(const void* x, const int32_t* positions, void* y, int64_t N, int64_t heads, int64_t head_channels,
               int64_t G, const int32_t* sections, int axes, double base, int64_t x_stride, int64_t y_stride,
               int inverse, int io_dtype, void* stream) {
    if (N < 0 || heads < 1 || head_channels < 1)
        return report(EQLIN_ERR_INVALID_ARG, "N must be >= 0, heads and head_channels >= 1");
    if (!known_dtype(io_dtype)) return report(EQLIN_ERR_INVALID_ARG, "unknown dtype");
    const int lg = log2_group(G);
    if (lg < 0) return report(EQLIN_ERR_UNSUPPORTED, "G must be 1, 2, 4, 8 or 16");
    if (head_channels % 2 || head_channels > 2 * rope::kMaxPairs)
        return report(EQLIN_ERR_UNSUPPORTED, "head_channels must be even and at most 256");
    if (!sections || axes < 1 || axes > rope::kMaxAxes)
        return report(EQLIN_ERR_INVALID_ARG, "sections is NULL or axes is not 1..4");
    if (!(base >= 1.0) || !std::isfinite(base)) return report(EQLIN_ERR_INVALID_ARG, "base must be finite and >= 1");
    int64_t total = 0;
    for (int a = 0; a < axes; ++a) {
        if (sections[a] < 0) return report(EQLIN_ERR_INVALID_ARG, "a section is negative");
        total += sections[a];
    }
    if (total != head_channels / 2)
        return report(EQLIN_ERR_INVALID_ARG, "the sections must add up to head_channels / 2 pairs");
    const int64_t width = head_channels * G;
    if (heads > (int64_t(1) << 16) || N >= (int64_t(1) << 31))
        return report(EQLIN_ERR_UNSUPPORTED, "at most 65536 heads and fewer than 2^31 tokens");
    if (x_stride < heads * width || y_stride < heads * width)
        return report(EQLIN_ERR_INVALID_ARG, "a row stride is smaller than heads * head_channels * G");
    if (x_stride > (int64_t(1) << 40) || y_stride > (int64_t(1) << 40))
        return report(EQLIN_ERR_INVALID_ARG, "a row stride is too large");
    if (N == 0) return EQLIN_OK;
    if (!x || !y || !positions) return report(EQLIN_ERR_INVALID_ARG, "x, y or positions is NULL");
    const int e = elem_bytes(io_dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(positions, 4))
        return report(EQLIN_ERR_MISALIGNED, "x, y or positions is not aligned to its element size");
    rope::Params p;
    p.half = static_cast<int>(width / 2);
    // widest vector that the head's halves, the row strides and the addresses allow
    int vec = 16 / e;
    while (vec > 1 && (p.half % vec || x_stride % vec || y_stride % vec || !aligned(x, size_t(vec) * e) ||
                       !aligned(y, size_t(vec) * e)))
        vec /= 2;
    int sms = 0, s;
    if ((s = current_device(nullptr, &sms)) != EQLIN_OK) return s;
    p.x = x;
    p.y = y;
    p.positions = positions;
    p.N = N;
    p.x_stride = x_stride;
    p.y_stride = y_stride;
    p.heads = static_cast<int>(heads);
    p.pairs = static_cast<int>(head_channels / 2);
    p.lg_g = lg;
    p.axes = axes;
    p.sign = inverse ? -1.f : 1.f;
    int j = 0;
    for (int a = 0; a < rope::kMaxAxes; ++a) {
        const int n = a < axes ? sections[a] : 0;
        for (int k = 0; k < n; ++k, ++j) {
            // base^(-k/n) radians per position, in turns, as a binary fraction of 64 bits
            const long double turns = powl(base, -static_cast<long double>(k) / n) / 6.283185307179586476925286766559L;
            p.turns[j] = static_cast<unsigned long long>(turns * 18446744073709551616.0L + 0.5L);
        }
        p.section_end[a] = j;
    }
    for (; j < rope::kMaxPairs; ++j) p.turns[j] = 0;
    // About kUnroll vectors for each thread of a block, fewer tokens where that leaves SMs
    // without a block.
    const int64_t per_token = heads * (p.half / vec);
    int64_t tokens = std::max<int64_t>(1, int64_t(rope::kThreads) * rope::kUnroll / per_token);
    tokens = std::min(tokens, std::max<int64_t>(1, N / (2 * sms)));
    tokens = std::min<int64_t>(tokens, rope::kMaxSmemPairs / p.pairs);
    p.tokens = static_cast<int>(tokens);
    const unsigned blocks = static_cast<unsigned>((N + tokens - 1) / tokens);
    const size_t smem = size_t(tokens) * p.pairs * sizeof(float2);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (io_dtype == EQLIN_F32) return launch_rope_vec<float>(vec, p, blocks, smem, st);
    if (io_dtype == EQLIN_F16) return launch_rope_vec<__half>(vec, p, blocks, smem, st);
    return launch_rope_vec<__nv_bfloat16>(vec, p, blocks, smem, st);
}

}  // extern "C"
