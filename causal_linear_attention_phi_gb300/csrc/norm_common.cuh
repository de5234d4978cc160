// norm_common.cuh -- pieces shared by the norm kernels: fp32 pairs, 16-byte vectors as pairs, sums over a row's threads.
#pragma once

#include "la_internal.cuh"
#include "sm100.cuh"

namespace la {
namespace norm {

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
          "l"(reinterpret_cast<const uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A vector of 16 bytes as float pairs, and back.
template <typename T>
struct Pairs;
template <>
struct Pairs<__nv_bfloat16> {
    static constexpr int n = 4;
    __device__ static void get(const void* p, float2 (&v)[4]) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        v[0] = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u));
        v[1] = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
        v[2] = make_float2(__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xFFFF0000u));
        v[3] = make_float2(__uint_as_float(w.w << 16), __uint_as_float(w.w & 0xFFFF0000u));
    }
    __device__ static void put(void* p, const float2 (&v)[4]) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(sm100::pack_bf16x2(v[0].x, v[0].y), sm100::pack_bf16x2(v[1].x, v[1].y),
                       sm100::pack_bf16x2(v[2].x, v[2].y), sm100::pack_bf16x2(v[3].x, v[3].y));
    }
};
template <>
struct Pairs<float> {
    static constexpr int n = 2;
    __device__ static void get(const void* p, float2 (&v)[2]) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        v[0] = make_float2(w.x, w.y);
        v[1] = make_float2(w.z, w.w);
    }
    __device__ static void put(void* p, const float2 (&v)[2]) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
};

// Sums of x over the TPR threads of a row, TPR <= 32 by shuffles, else over the row's warps by a barrier of its own
// (id 1 + row of the block) and `buf` (two halves taken in turn).
template <int TPR, int NV, int W8>
__device__ __forceinline__ void group_sum(float (&x)[NV], float (*buf)[W8], int group, int t, int& turn) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        float(*half)[W8] = buf + NV * turn;
        turn ^= 1;
        if ((t & 31) == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i) half[i][t >> 5] = x[i];
        sm100::named_barrier(1 + group, TPR);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) x[i] += half[i][w];
        }
    }
}

}  // namespace norm
}  // namespace la
