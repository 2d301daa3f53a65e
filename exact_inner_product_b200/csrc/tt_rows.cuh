// tt_rows.cuh - rows of fp32 or bf16 numbers as fp32 registers: chunks of E
// consecutive elements per load or store, and sums over a group of lanes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace tt {

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float* x) {
    x[0] = __uint_as_float(w << 16);
    x[1] = __uint_as_float(w & 0xFFFF0000u);
}

// E consecutive elements at p as they lie in memory (16-byte pieces where E
// allows), so that loads can be held in registers before they are unpacked.
// p is aligned to min(16, E * sizeof(T)) bytes.
template <typename T, int E>
struct Raw;

template <>
struct Raw<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
template <>
struct Raw<float, 4> {
    float4 a;
    __device__ __forceinline__ void load(const float* p) { a = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float* x) const { x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w; }
};
template <>
struct Raw<float, 2> {
    float2 a;
    __device__ __forceinline__ void load(const float* p) { a = __ldg(reinterpret_cast<const float2*>(p)); }
    __device__ __forceinline__ void zero() { a = make_float2(0.f, 0.f); }
    __device__ __forceinline__ void get(float* x) const { x[0] = a.x, x[1] = a.y; }
};
template <>
struct Raw<float, 1> {
    float a;
    __device__ __forceinline__ void load(const float* p) { a = __ldg(p); }
    __device__ __forceinline__ void zero() { a = 0.f; }
    __device__ __forceinline__ void get(float* x) const { x[0] = a; }
};
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float* x) const {
        unpack_bf16x2(a.x, x), unpack_bf16x2(a.y, x + 2), unpack_bf16x2(a.z, x + 4), unpack_bf16x2(a.w, x + 6);
    }
};
template <>
struct Raw<__nv_bfloat16, 4> {
    uint2 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void zero() { a = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float* x) const { unpack_bf16x2(a.x, x), unpack_bf16x2(a.y, x + 2); }
};
template <>
struct Raw<__nv_bfloat16, 2> {
    uint32_t a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint32_t*>(p)); }
    __device__ __forceinline__ void zero() { a = 0u; }
    __device__ __forceinline__ void get(float* x) const { unpack_bf16x2(a, x); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
    unsigned short a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        a = __ldg(reinterpret_cast<const unsigned short*>(p));
    }
    __device__ __forceinline__ void zero() { a = 0; }
    __device__ __forceinline__ void get(float* x) const { x[0] = __uint_as_float((uint32_t)a << 16); }
};

// E fp32 values to p, rounded to nearest-even where T is bf16.
template <int E>
__device__ __forceinline__ void store_row(float* p, const float* x) {
    if constexpr (E == 1) {
        *p = x[0];
    } else if constexpr (E == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
}
template <int E>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float* x) {
    if constexpr (E == 1) {
        *p = __float2bfloat16_rn(x[0]);
    } else if constexpr (E == 2) {
        *reinterpret_cast<uint32_t*>(p) = bf16x2_bits(x[0], x[1]);
    } else if constexpr (E == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]));
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]),
                                                  bf16x2_bits(x[4], x[5]), bf16x2_bits(x[6], x[7]));
    }
}

// Sum over the L lanes (a power of two) that share a row; every lane gets it.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace tt
