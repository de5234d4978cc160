// cross_step.cu -- cross attention of a few queries to a kept state: out = phi(q)^T S / phi(q)^T z for the rows of
// queries that share a head of keys (one token of each of its heads of queries, or a few tokens).
//
// Bound by memory: a state of Dk x Dv fp32 is read once, everything else is O(Dk + Dv) to a row.  A block owns a head, or 64 columns of
// one (32 KB: five blocks to an SM take over from one another more evenly than two with 64 KB): its threads issue all loads of S before any arithmetic and keep S in registers (at most 16 16-byte vectors each),
// so that every further row costs shared memory and arithmetic only.  Rows are taken kRows at a time: each thread
// forms their partial sums over its rows of S, and the warps' sums are joined in shared memory in a fixed order.
#include "cross.cuh"

namespace la {
namespace cross {
namespace {

// DV: the columns of a block.
template <int DK, int DV>
struct Few {
    static constexpr int kVecs = DK * DV / 4;
    static constexpr int kThreads = kVecs / 8 < 32 ? 32 : kVecs / 8 > 256 ? 256 : kVecs / 8;
    static constexpr int kWarps = kThreads / 32;
    static constexpr int kCols = DV / 4;                 // 16-byte vectors of a row of S
    static constexpr int kPer = kThreads / kCols;        // rows of S in one load of the block
    static constexpr int kHeld = kVecs / kThreads;       // vectors held by a thread
};

template <typename T, int DK, int DV, int kRows>
__global__ void __launch_bounds__(Few<DK, DV>::kThreads)
cross_few_kernel(const T* __restrict__ q, const float* __restrict__ S, const float* __restrict__ z, T* __restrict__ o,
                 int R, int pitch) {
    using F = Few<DK, DV>;
    __shared__ float ph[kRows][DK];
    __shared__ __align__(16) float part[F::kWarps][kRows][DV];
    __shared__ float inv[kRows], zs[DK];
    __shared__ bool keys[kRows];
    pdl_enter();  // launched with programmatic dependent launch
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c4 = tid % F::kCols, r0 = tid / F::kCols;
    const size_t bh = blockIdx.y;
    const float* Sh = S + bh * DK * pitch + blockIdx.x * DV;
    const float* zh = z + bh * DK;
    float4 s[F::kHeld];
#pragma unroll
    for (int x = 0; x < F::kHeld; ++x)
        s[x] = *reinterpret_cast<const float4*>(Sh + (size_t)(r0 + F::kPer * x) * pitch + 4 * c4);
    // z and the first rows of q are on their way together with S: loads one after another were three latencies to a block
    constexpr int kZ = (DK + F::kThreads - 1) / F::kThreads, kQ = (kRows * DK + F::kThreads - 1) / F::kThreads;
    const T* qh = q + bh * R * DK;
    float zr[kZ], qr[kQ];
    auto fetch_q = [&](int base) {
        const int all = min(kRows, R - base) * DK;
#pragma unroll
        for (int x = 0; x < kQ; ++x) qr[x] = tid + x * F::kThreads < all ? to_f32(qh[(size_t)base * DK + tid + x * F::kThreads]) : 0.f;
    };
    fetch_q(0);
#pragma unroll
    for (int x = 0; x < kZ; ++x) zr[x] = tid + x * F::kThreads < DK ? zh[tid + x * F::kThreads] : 0.f;
#pragma unroll
    for (int x = 0; x < kZ; ++x)
        if (tid + x * F::kThreads < DK) zs[tid + x * F::kThreads] = zr[x];
    T* oh = o + bh * R * pitch + blockIdx.x * DV;
    for (int base = 0; base < R; base += kRows) {
        const int n = min(kRows, R - base);
#pragma unroll
        for (int x = 0; x < kQ; ++x)
            if (tid + x * F::kThreads < n * DK) (&ph[0][0])[tid + x * F::kThreads] = phi_of(qr[x]);
        __syncthreads();
        if (base + kRows < R) fetch_q(base + kRows);
        for (int r = warp; r < n; r += F::kWarps) {
            float den = 0.f;
            bool some = false;
            for (int d = lane; d < DK; d += 32) {
                den = fmaf(ph[r][d], zs[d], den);
                some = some || zs[d] != 0.f;
            }
#pragma unroll
            for (int y = 16; y > 0; y >>= 1) den += __shfl_xor_sync(0xffffffffu, den, y);
            some = __any_sync(0xffffffffu, some);  // the head has keys
            if (lane == 0) inv[r] = over(den), keys[r] = some;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= n) break;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < F::kHeld; ++x) {
                const float p = ph[r][r0 + F::kPer * x];
                a.x = fmaf(p, s[x].x, a.x);
                a.y = fmaf(p, s[x].y, a.y);
                a.z = fmaf(p, s[x].z, a.z);
                a.w = fmaf(p, s[x].w, a.w);
            }
#pragma unroll
            for (int y = F::kCols; y < 32; y <<= 1) {  // lanes of the same columns
                a.x += __shfl_xor_sync(0xffffffffu, a.x, y);
                a.y += __shfl_xor_sync(0xffffffffu, a.y, y);
                a.z += __shfl_xor_sync(0xffffffffu, a.z, y);
                a.w += __shfl_xor_sync(0xffffffffu, a.w, y);
            }
            if (lane < F::kCols) *reinterpret_cast<float4*>(&part[warp][r][4 * c4]) = a;
        }
        __syncthreads();
        for (int x = tid; x < n * DV; x += F::kThreads) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < F::kWarps; ++w) a += part[w][x / DV][x % DV];
            if (LA_DCHECK(base + x / DV < R)) oh[(size_t)(base + x / DV) * pitch + x % DV] = from_f32<T>(keys[x / DV] ? a * inv[x / DV] : 0.f);
        }
        __syncthreads();  // before the next rows
    }
}

template <typename T, int DK, int DV>
cudaError_t go(const void* q, const float* S, const float* z, void* o, int heads, int R, cudaStream_t st) {
    constexpr int kCols = DV < 64 ? DV : 64;
    auto kern = R == 1   ? cross_few_kernel<T, DK, kCols, 1>
                : R == 2 ? cross_few_kernel<T, DK, kCols, 2>
                         : cross_few_kernel<T, DK, kCols, 4>;
    launch_begin("cross_few", st);
    const cudaError_t e = launch_pdl(kern, dim3(DV / kCols, heads), dim3(Few<DK, kCols>::kThreads), 0, st, (const T*)q, S, z, (T*)o, R, DV);
    const cudaError_t e2 = launch_end("cross_few", st);
    return e != cudaSuccess ? e : e2;
}

template <typename T>
cudaError_t pick(const void* q, const float* S, const float* z, void* o, const la_cross_shape& s, cudaStream_t st) {
    const int heads = s.B * s.Hk, R = (int)query_rows(s);
#define LA_FEW(a, b) \
    if (s.Dk == a && s.Dv == b) return go<T, a, b>(q, S, z, o, heads, R, st);
#define LA_FEW4(a) LA_FEW(a, 16) LA_FEW(a, 32) LA_FEW(a, 64) LA_FEW(a, 128)
    LA_FEW4(16) LA_FEW4(32) LA_FEW4(64) LA_FEW4(128)
#undef LA_FEW4
#undef LA_FEW
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t apply_few(const void* q, const float* S, const float* z, void* o, const la_cross_shape& s, cudaStream_t st) {
    return s.dtype == LA_BF16 ? pick<__nv_bfloat16>(q, S, z, o, s, st) : pick<float>(q, S, z, o, s, st);
}

}  // namespace cross
}  // namespace la
