// eqlin_vec.cuh -- vectors of I/O elements as fp32 registers, for the memory-bound kernels:
// VEC consecutive elements move as one load or store of VEC * sizeof(T) <= 16 bytes.
#pragma once

#include <cstdint>

#include "io16.cuh"

namespace eqlin {

template <int BYTES>
struct RawVec;
template <>
struct RawVec<16> { using type = uint4; };
template <>
struct RawVec<8> { using type = uint2; };
template <>
struct RawVec<4> { using type = uint32_t; };
template <>
struct RawVec<2> { using type = uint16_t; };

template <class T, int VEC>
struct Vec {
    using Raw = typename RawVec<VEC * sizeof(T)>::type;
    // Raw words and their elements: load() and store() only move, unpack() and pack() convert.
    __device__ __forceinline__ static Raw load(const T* p) { return *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ static void store(T* p, const Raw& r) { *reinterpret_cast<Raw*>(p) = r; }
    __device__ __forceinline__ static void unpack(const Raw& r, float (&v)[VEC]) {
        if constexpr (sizeof(T) == 4) {
            const float* f = reinterpret_cast<const float*>(&r);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = f[i];
        } else if constexpr (VEC == 1) {
            v[0] = Io16<T>::lo(r);
        } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                v[2 * i] = Io16<T>::lo(w[i]);
                v[2 * i + 1] = Io16<T>::hi(w[i]);
            }
        }
    }
    __device__ __forceinline__ static Raw pack(const float (&v)[VEC]) {
        Raw r;
        if constexpr (sizeof(T) == 4) {
            float* f = reinterpret_cast<float*>(&r);
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = v[i];
        } else if constexpr (VEC == 1) {
            r = static_cast<uint16_t>(Io16<T>::pack(v[0], 0.f) & 0xFFFFu);
        } else {
            uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) w[i] = Io16<T>::pack(v[2 * i], v[2 * i + 1]);
        }
        return r;
    }
};

// One parameter value of any I/O type (dtype as in eqlin_dtype: 0 fp32, 1 bf16, 2 fp16).
__device__ __forceinline__ float load_param(const void* p, int dtype, long long i) {
    if (dtype == 0) return static_cast<const float*>(p)[i];
    const uint16_t h = static_cast<const uint16_t*>(p)[i];
    return dtype == 1 ? Io16<__nv_bfloat16>::lo(h) : Io16<__half>::lo(h);
}

}  // namespace eqlin
