// tc_cross.cuh -- shared pieces of the tensor-core (tcgen05 / TMEM / TMA) kernels of cross attention, bf16 heads.
//
// Heads are padded on chip to KB (keys) and VB (values) blocks of 64 columns by the tile copies, which fill what lies
// outside a tensor with zeros.  A tile of `rows` rows is KB or VB blocks of rows x 128 bytes with the 128-byte
// swizzle: 16-byte chunk lc of row r of a block sits at chunk lc ^ (r & 7).
//
// The state (S, z), and (R, r) of the gradient, pass between kernels as an image: S as two bf16 parts (hi, then lo =
// S - hi), each a swizzled tile of 64 KB rows by VB blocks as the products' operands want it, then z as 64 KB floats; a
// block brings it into shared memory with one copy.  Behind them 64 VB floats: what a centred image has taken out of S.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "cross.cuh"
#include "norm_common.cuh"
#include "shared_memory.cuh"
#include "tc_common.cuh"

namespace la {
namespace cross {

using namespace sm100;

constexpr int kSumRows = 64;   // rows of a chunk of the sums
constexpr int kRowChunk = 128; // rows of a chunk of the queries, and of the keys in the gradient

constexpr size_t image_part(int KB, int VB) { return (size_t)KB * VB * 8192; }
constexpr size_t image_bytes(int KB, int VB) { return 2 * image_part(KB, VB) + (size_t)(KB + VB) * 256; }
#ifdef __CUDACC__
template <typename C>  // char or const char
__device__ __forceinline__ auto image_centre(C* image, int KB, int VB) {
    using F = std::conditional_t<std::is_const_v<C>, const float, float>;
    return reinterpret_cast<F*>(image + 2 * image_part(KB, VB) + (size_t)KB * 256);
}
#endif
// A record of the sums: 128 accumulator rows of 64 VB floats, 128 floats of z (KB = 1: the upper 64 of either belong to the
// lo parts and are added to the lower).
constexpr size_t record_floats(int VB) { return (size_t)128 * 64 * VB + 128; }

// Stages of a ring that two groups take in turn: an even number, so that a stage is always the same group's, which then waits
// for each of its phases (a wait that skips one can be let through by the phase before).
constexpr int even_stages(int fit, int most) { return (fit < most ? fit : most) / 2 * 2; }

inline int blocks64(int d) { return d > 64 ? 2 : 1; }

__device__ __forceinline__ int swz(int row, int lc) { return row * 128 + (((lc & 7) ^ (row & 7)) << 4); }
// Operand descriptors: a tile's first, and steps from it added to its address field (shared memory ends below the field's).
// K-major operand, 16-element step kk: blocks of 64 elements are `block` bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int kk, uint32_t block) {
    return smem_desc_sw128(tile, 16, 1024) + (((kk >> 2) * block + (kk & 3) * 32) >> 4);
}
// MN-major operand, 16-row step kk: blocks of 64 M or N elements are `block` bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int kk, uint32_t block) {
    return smem_desc_sw128(tile, block, 1024) + ((kk * 2048) >> 4);
}

// A bounded wait whose outcome is the same for a whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, LA_ERR_TIMEOUT));
}

// One arrival for a warp, after all its lanes have got here (32 arrivals of lanes are 32 turns at the barrier's word).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The products are issued by one thread, but a whole warp goes through the loop around them: operands of tcgen05.mma are
// uniform registers, which code that one lane runs alone has to fill one by one before each product (about 130 cycles a
// product, which bound all four kernels).  `uniform` tells the compiler that all lanes hold the same value.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// Debug build: a tile copy of a [heads][rows][D] tensor.
__device__ __forceinline__ void check_copy(int x, int row, int rows, int bh, int heads) {
    LA_DCHECK((x == 0 || x == 64) && row >= 0 && row < rows && bh >= 0 && bh < heads);
}

// Whether a head has keys, from its z in shared memory.  A whole warp.
template <int KB>
__device__ __forceinline__ bool any_key(const float* zs) {
    bool some = false;
#pragma unroll
    for (int x = 0; x < 2 * KB; ++x) some = some || zs[32 * x + (threadIdx.x & 31)] != 0.f;
    return __any_sync(0xffffffffu, some);
}

__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(tc::bf_lo(w), tc::bf_hi(w)); }
// phi of a pair of bf16, as phi_of: the bounds by 0 are exact in bf16, both in one instruction, and the upper one is added as it
// is, without conversion (sums over 128 x 64 heads 54.0 us with bounds in fp32, 52.7 so; bounds and conversions share a pipe).
__device__ __forceinline__ float2 phi2(uint32_t w) {
    uint32_t low, high;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(low) : "r"(w), "r"(0u));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(high) : "r"(w), "r"(0u));
    const float2 t = norm::mul2(unpack2(low), norm::both(1.4426950408889634f));
    float2 p;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "add.f32.bf16 %0, l, %3;\n\t"
        "add.f32.bf16 %1, h, %4;\n\t}"
        : "=f"(p.x), "=f"(p.y)
        : "r"(high), "f"(ex2_approx(t.x)), "f"(ex2_approx(t.y)));
    return p;
}
__device__ __forceinline__ uint32_t pack2(float2 x) { return pack_bf16x2(x.x, x.y); }
// hi and lo bf16 parts of two floats.
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
    hi = pack2(x);
    lo = pack2(norm::fma2(unpack2(hi), norm::both(-1.f), x));
}

// host
struct TcLayout {
    size_t rec, S, R, bytes;  // records; images of (S, z) and of (R, r)
    int sum_ctas, query_ctas, key_ctas;
};
TcLayout tc_layout(const la_cross_shape& s, int op);

// Records of the heads, or a caller's state, to images; with S_out the sums also as fp32 state.  kState: the forward's, (S, z) as
// they are; kCentred: the gradient's; kGradSums: (R, r) of sums formed with the centred images `centre`.
enum JoinMode { kState, kCentred, kGradSums };
cudaError_t tc_join(JoinMode mode, const float* rec, const float* S, const float* z, char* image, const char* centre, float* S_out,
                    float* z_out, const Rows& rows, int chunk, int ctas, const la_cross_shape& s, cudaStream_t st);
cudaError_t tc_sums(const void* k, const void* v, const Rows& keys, float* rec, int ctas, const la_cross_shape& s, cudaStream_t st);

// A kernel that takes nearly all of an SM's shared memory: opted in once for its one size.
template <typename K, typename... A>
cudaError_t tc_run(const char* name, K kern, dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    launch_begin(name, st);
    e = launch_pdl(kern, grid, dim3(threads), smem, st, args...);
    const cudaError_t e2 = launch_end(name, st);
    return e != cudaSuccess ? e : e2;
}

}  // namespace cross
}  // namespace la
