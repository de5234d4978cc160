// layer_norm.cu -- layer norm over the last dimension, forward and gradient:
//   y = (x - mean) rstd w + b,   mean = sum x / C,   rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   dx = rstd (d - sum d / C - h sum(d h) / C),  d = dy w,  h = (x - mean) rstd;   dw = sum_rows dy h,  db = sum_rows dy
//
// Bound by memory: each element is read once and written once.  A row stays on chip between its passes, so the variance
// is the mean of squared differences from the mean, not a difference of sums.  Rows that 16-byte vectors divide are
// streamed through shared memory (ln_fwd_tiles, and ln_bwd_tiles up to 4096 elements); the others are held in the
// registers of TPR threads (ln_fwd_kernel, ln_bwd_kernel).  The gradient's blocks walk rows and keep dw and db of
// their columns in registers; each block writes its sums once and a second kernel adds the blocks' sums in
// a fixed order (no atomics: the same bits every time).  Statistics and sums are fp32; products and fused
// multiply-adds are written out, so a call gives the same bits with and without the statistics returned.
// Measured on one GB300, of the 6.76 TB/s a copy reaches: forward 131072 x 2048 bf16 178 us (0.89), gradient
// 1048576 x 128 bf16 131 us (0.92).
#include "layer_norm.cuh"
#include "sm100.cuh"

namespace la {
namespace ln {
namespace {

constexpr int kBlock = 256;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
    T e[VEC];
};

// Sum of x over the TPR threads of a row; with TPR > 32 the block is one row and `buf` (2 x 32 floats, the halves
// taken in turn) joins its warps.
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&x)[NV], float (*buf)[32], int& turn) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    if (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        float(*half)[32] = buf + NV * turn;
        turn ^= 1;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i) half[i][warp] = x[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float s = lane < W ? half[i][lane] : 0.f;
#pragma unroll
            for (int o = (W < 32 ? W : 32) / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            x[i] = __shfl_sync(0xffffffffu, s, 0);
        }
    }
}

template <typename T, int VPT, int TPR>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock)
ln_fwd_kernel(const T* x, const T* __restrict__ w, const T* __restrict__ b, T* y,
              float* __restrict__ mean, float* __restrict__ rstd, long long rows, int C, float eps) {
    __shared__ float buf[2][32];
    pdl_enter();  // launched with programmatic dependent launch
    constexpr int kRows = TPR > 32 ? 1 : kBlock / TPR;  // rows of a block
    const int t = threadIdx.x % TPR, sub = TPR > 32 ? 0 : threadIdx.x / TPR;
    const float inv = 1.f / (float)C;
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * kRows; r0 < rows; r0 += (long long)gridDim.x * kRows) {
        const long long r = r0 + sub;
        const bool in = r < rows;
        const T* xr = x + r * C;
        float xv[VPT];
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && t + TPR * i < C) xv[i] = to_f32(xr[t + TPR * i]);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && t + TPR * i < C) s[0] += xv[i];
        row_sum<TPR, 1>(s, buf, turn);
        const float mu = __fmul_rn(s[0], inv);
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && t + TPR * i < C) {
                const float d = xv[i] - mu;
                s[0] = fmaf(d, d, s[0]);
            }
        row_sum<TPR, 1>(s, buf, turn);
        const float rs = 1.f / sqrtf(fmaf(s[0], inv, eps));
        if (in && t == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = t + TPR * i;
            if (!in || c >= C) continue;
            const float h = __fmul_rn(xv[i] - mu, rs);
            y[r * C + c] = from_f32<T>(fmaf(h, w ? to_f32(w[c]) : 1.f, b ? to_f32(b[c]) : 0.f));
        }
    }
}

// Block partial sums: part[block][2][C] (dw, then db); null without a weight gradient.
template <typename T, int VEC, int VPT, int TPR>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock)
ln_bwd_kernel(const T* x, const T* __restrict__ w, const float* __restrict__ mean,
              const float* __restrict__ rstd, const T* dy, T* dx, float* __restrict__ part,
              long long rows, int C) {
    using V = Vec<T, VEC>;
    __shared__ float buf[4][32];
    extern __shared__ float sums[];  // [kRows][C], where a block holds several rows
    pdl_enter();                     // launched with programmatic dependent launch
    constexpr int kRows = TPR > 32 ? 1 : kBlock / TPR;
    const int t = threadIdx.x % TPR, sub = TPR > 32 ? 0 : threadIdx.x / TPR, nv = C / VEC;
    const float inv = 1.f / (float)C;
    int turn = 0;
    float dw[VPT * VEC], db[VPT * VEC];
#pragma unroll
    for (int i = 0; i < VPT * VEC; ++i) dw[i] = db[i] = 0.f;
    for (long long r0 = (long long)blockIdx.x * kRows; r0 < rows; r0 += (long long)gridDim.x * kRows) {
        const long long r = r0 + sub;
        const bool in = r < rows;
        V xv[VPT], dv[VPT];
        const float mu = in ? mean[r] : 0.f, rs = in ? rstd[r] : 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && t + TPR * i < nv) {
                xv[i] = reinterpret_cast<const V*>(x + r * C)[t + TPR * i];
                dv[i] = reinterpret_cast<const V*>(dy + r * C)[t + TPR * i];
            }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = t + TPR * i;
            if (!in || c >= nv) continue;
            V wv;
            if (w) wv = reinterpret_cast<const V*>(w)[c];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float g = to_f32(dv[i].e[e]), h = __fmul_rn(to_f32(xv[i].e[e]) - mu, rs);
                const float d = w ? __fmul_rn(g, to_f32(wv.e[e])) : g;
                s[0] += d;
                s[1] = fmaf(d, h, s[1]);
                dw[i * VEC + e] = fmaf(g, h, dw[i * VEC + e]);
                db[i * VEC + e] += g;
            }
        }
        row_sum<TPR, 2>(s, buf, turn);
        const float m0 = __fmul_rn(s[0], inv), m1 = __fmul_rn(s[1], inv);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = t + TPR * i;
            if (!in || c >= nv) continue;
            V wv, o;
            if (w) wv = reinterpret_cast<const V*>(w)[c];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float g = to_f32(dv[i].e[e]), h = __fmul_rn(to_f32(xv[i].e[e]) - mu, rs);
                const float d = w ? __fmul_rn(g, to_f32(wv.e[e])) : g;
                o.e[e] = from_f32<T>(rs * fmaf(-h, m1, d - m0));
            }
            reinterpret_cast<V*>(dx + r * C)[c] = o;
        }
    }
    if (!part) return;
    float* p = part + (size_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float* acc = which ? db : dw;
        if (kRows == 1) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (t + TPR * i < nv)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) p[which * C + (t + TPR * i) * VEC + e] = acc[i * VEC + e];
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (t + TPR * i < nv)
#pragma unroll
                for (int e = 0; e < VEC; ++e) sums[sub * C + (t + TPR * i) * VEC + e] = acc[i * VEC + e];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += kBlock) {
            float v = 0.f;
            for (int y = 0; y < kRows; ++y) v += sums[y * C + c];
            p[which * C + c] = v;
        }
    }
}

// ------------------------------------------------------------------ streamed rows (16-byte vectors divide a row)
// Rows are contiguous, so a tile of them is one bulk copy.  A block keeps two or three tiles in flight in shared memory, which
// is what it takes to keep the memory busy (about 50 KB an SM); rows held in registers instead, with a barrier between
// load and use, reached 0.74 of the copy rate forward (131072 x 2048 bf16; here 0.89) and 0.68 in the gradient
// (1048576 x 128; here 0.92).  What is left is the drain of the last tiles and the statistics.
constexpr int kFwdStages = 2, kBwdStages = 3;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            sm100::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
        : "memory");
}
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
template <int TPR, int NV>
__device__ __forceinline__ void group_sum(float (&x)[NV], float (*buf)[8], int group, int t, int& turn) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        float(*half)[8] = buf + NV * turn;
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

// After a wait that ran out: wait once more, with the same limit, for the copies in flight (none is left behind).
template <int kStages>
__device__ __noinline__ void drain(uint64_t* bar, long long issued, int* err) {
    for (long long i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
        sm100::mbar_wait(bar + i % kStages, (int)(i / kStages) & 1, err, LA_ERR_TIMEOUT);
}

struct Tiles {
    long long rows, tiles;
    int C, R;       // R rows to a tile
    uint32_t row;   // bytes of a row
};

// kBlock threads; TPR threads to a row, kBlock / TPR rows at a time.
template <typename T, int TPR>
__global__ void __launch_bounds__(kBlock)
ln_fwd_tiles(const T* x, const T* __restrict__ w, const T* __restrict__ b, T* y, float* __restrict__ mean,
             float* __restrict__ rstd, Tiles tl, float eps, int* err) {
    using P = Pairs<T>;
    constexpr int VEC = 16 / (int)sizeof(T), kRows = kBlock / TPR;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bar[kFwdStages];
    __shared__ float buf[kRows][2][8];
    const int tid = threadIdx.x, t = tid % TPR, sub = tid / TPR, nv = tl.C / VEC;
    const uint32_t tile = tl.row * tl.R;
    if (tid == 0) {
        for (int s = 0; s < kFwdStages; ++s) sm100::mbar_init(bar + s, 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();  // launched with programmatic dependent launch
    auto rows_of = [&](long long k) { return (int)min((long long)tl.R, tl.rows - k * tl.R); };
    bool ok = true;
    long long issued = 0;
    auto load = [&](long long i) {  // the i-th tile of this block
        const long long k = blockIdx.x + i * gridDim.x;
        if (tid != 0 || k >= tl.tiles || !ok) return;
        issued = i + 1;
        const int s = (int)(i % kFwdStages);
        const uint32_t bytes = rows_of(k) * tl.row;
        sm100::mbar_arrive_expect_tx(bar + s, bytes);
        bulk_load(smem + s * tile, reinterpret_cast<const uint8_t*>(x) + k * tile, bytes, bar + s);
    };
    for (int i = 0; i < kFwdStages; ++i) load(i);
    const float inv = 1.f / (float)tl.C;
    int turn = 0;
    long long i = 0;
    for (long long k = blockIdx.x; k < tl.tiles; k += gridDim.x, ++i) {
        const int s = (int)(i % kFwdStages), n = rows_of(k);
        ok = ok && sm100::mbar_wait(bar + s, (int)(i / kFwdStages) & 1, err, LA_ERR_TIMEOUT);
        __syncwarp();
        for (int r0 = 0; r0 < n; r0 += kRows) {
            const int r = r0 + sub;
            const bool in = r < n;  // the same for a whole warp where a row has a barrier
            if (TPR > 32 && !in) break;
            const uint8_t* xr = smem + s * tile + (in ? r : 0) * tl.row;
            float2 v[P::n], a2 = both(0.f);
#pragma unroll 4
            for (int c = t; c < nv; c += TPR) {
                P::get(xr + 16 * c, v);
#pragma unroll
                for (int e = 0; e < P::n; ++e) a2 = add2(a2, v[e]);
            }
            float a[1] = {a2.x + a2.y};
            group_sum<TPR, 1>(a, buf[sub], sub, t, turn);
            const float mu = __fmul_rn(a[0], inv);
            a2 = both(0.f);
#pragma unroll 4
            for (int c = t; c < nv; c += TPR) {
                P::get(xr + 16 * c, v);
#pragma unroll
                for (int e = 0; e < P::n; ++e) {
                    const float2 d = add2(v[e], both(-mu));
                    a2 = fma2(d, d, a2);
                }
            }
            a[0] = a2.x + a2.y;
            group_sum<TPR, 1>(a, buf[sub], sub, t, turn);
            const float rs = 1.f / sqrtf(fmaf(a[0], inv, eps));
            const long long row = k * tl.R + r;
            if (in && t == 0) {
                if (mean) mean[row] = mu;
                if (rstd) rstd[row] = rs;
            }
            if (!in) continue;
            uint8_t* yr = reinterpret_cast<uint8_t*>(y) + row * tl.row;
#pragma unroll 4
            for (int c = t; c < nv; c += TPR) {
                float2 wv[P::n], bv[P::n];
                P::get(xr + 16 * c, v);
                if (w) P::get(reinterpret_cast<const uint4*>(w) + c, wv);
                if (b) P::get(reinterpret_cast<const uint4*>(b) + c, bv);
#pragma unroll
                for (int e = 0; e < P::n; ++e) {
                    const float2 h = mul2(add2(v[e], both(-mu)), both(rs));
                    v[e] = fma2(h, w ? wv[e] : both(1.f), b ? bv[e] : both(0.f));
                }
                P::put(yr + 16 * c, v);
            }
        }
        __syncthreads();  // the tile has been read
        load(i + kFwdStages);
    }
    if (!ok) drain<kFwdStages>(bar, issued, err);
}

// The gradient: x and dy tiles; a thread keeps dw and db of its columns (VPT vectors).
template <typename T, int VPT, int TPR>
__global__ void __launch_bounds__(kBlock)
ln_bwd_tiles(const T* x, const T* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
             const T* dy, T* dx, float* __restrict__ part, Tiles tl, int* err) {
    using P = Pairs<T>;
    constexpr int VEC = 16 / (int)sizeof(T), kRows = kBlock / TPR;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bar[kBwdStages];
    __shared__ float buf[kRows][4][8];
    const int tid = threadIdx.x, t = tid % TPR, sub = tid / TPR, nv = tl.C / VEC;
    const uint32_t tile = tl.row * tl.R;
    if (tid == 0) {
        for (int s = 0; s < kBwdStages; ++s) sm100::mbar_init(bar + s, 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();  // launched with programmatic dependent launch
    auto rows_of = [&](long long k) { return (int)min((long long)tl.R, tl.rows - k * tl.R); };
    bool ok = true;
    long long issued = 0;
    auto load = [&](long long i) {
        const long long k = blockIdx.x + i * gridDim.x;
        if (tid != 0 || k >= tl.tiles || !ok) return;
        issued = i + 1;
        const int s = (int)(i % kBwdStages);
        const uint32_t bytes = rows_of(k) * tl.row;
        sm100::mbar_arrive_expect_tx(bar + s, 2 * bytes);
        bulk_load(smem + 2 * s * tile, reinterpret_cast<const uint8_t*>(x) + k * tile, bytes, bar + s);
        bulk_load(smem + (2 * s + 1) * tile, reinterpret_cast<const uint8_t*>(dy) + k * tile, bytes, bar + s);
    };
    for (int i = 0; i < kBwdStages; ++i) load(i);
    float2 wv[VPT][P::n], dw[VPT][P::n], db[VPT][P::n];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int e = 0; e < P::n; ++e) {
            wv[i][e] = both(1.f);
            dw[i][e] = db[i][e] = both(0.f);
        }
        if (w && t + TPR * i < nv) P::get(reinterpret_cast<const uint4*>(w) + t + TPR * i, wv[i]);
    }
    const float inv = 1.f / (float)tl.C;
    int turn = 0;
    long long i = 0;
    // the statistics of this thread's next row, loaded a turn ahead
    float mu_next = 0.f, rs_next = 0.f;
    auto stats = [&](long long k, int r) {
        if (k < tl.tiles && r < rows_of(k)) {
            mu_next = mean[k * tl.R + r];
            rs_next = rstd[k * tl.R + r];
        }
    };
    stats(blockIdx.x, sub);
    for (long long k = blockIdx.x; k < tl.tiles; k += gridDim.x, ++i) {
        const int s = (int)(i % kBwdStages), n = rows_of(k);
        ok = ok && sm100::mbar_wait(bar + s, (int)(i / kBwdStages) & 1, err, LA_ERR_TIMEOUT);
        __syncwarp();
        for (int r0 = 0; r0 < n; r0 += kRows) {
            const int r = r0 + sub;
            const bool in = r < n;
            const float mu = mu_next, rs = rs_next;
            if (r0 + kRows < n)
                stats(k, r + kRows);
            else
                stats(k + gridDim.x, sub);
            if (TPR > 32 && !in) break;
            const long long row = k * tl.R + (in ? r : 0);
            const uint8_t* xr = smem + 2 * s * tile + (in ? r : 0) * tl.row;
            const uint8_t* dr = xr + tile;
            float2 s0 = both(0.f), s1 = s0;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = t + TPR * j;
                if (!in || c >= nv) continue;
                float2 xv[P::n], gv[P::n];
                P::get(xr + 16 * c, xv);
                P::get(dr + 16 * c, gv);
#pragma unroll
                for (int e = 0; e < P::n; ++e) {
                    const float2 h = mul2(add2(xv[e], both(-mu)), both(rs)), d = mul2(gv[e], wv[j][e]);
                    s0 = add2(s0, d);
                    s1 = fma2(d, h, s1);
                    dw[j][e] = fma2(gv[e], h, dw[j][e]);
                    db[j][e] = add2(db[j][e], gv[e]);
                }
            }
            float a[2] = {s0.x + s0.y, s1.x + s1.y};
            group_sum<TPR, 2>(a, buf[sub], sub, t, turn);
            if (!in) continue;
            const float2 m0 = both(-__fmul_rn(a[0], inv)), m1 = both(-__fmul_rn(a[1], inv));
            uint8_t* o = reinterpret_cast<uint8_t*>(dx) + row * tl.row;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = t + TPR * j;
                if (c >= nv) continue;
                float2 xv[P::n], gv[P::n];
                P::get(xr + 16 * c, xv);
                P::get(dr + 16 * c, gv);
#pragma unroll
                for (int e = 0; e < P::n; ++e) {
                    const float2 h = mul2(add2(xv[e], both(-mu)), both(rs)), d = mul2(gv[e], wv[j][e]);
                    gv[e] = mul2(fma2(h, m1, add2(d, m0)), both(rs));
                }
                P::put(o + 16 * c, gv);
            }
        }
        __syncthreads();  // the tiles have been read
        load(i + kBwdStages);
    }
    if (!ok) drain<kBwdStages>(bar, issued, err);
    if (!part) return;
    // the rows of a block joined in shared memory (the tiles are done with), then one record per block
    float* sums = reinterpret_cast<float*>(smem);
    float* p = part + (size_t)blockIdx.x * 2 * tl.C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = t + TPR * j;
            if (c >= nv) continue;
#pragma unroll
            for (int e = 0; e < P::n; ++e)
                *reinterpret_cast<float2*>(sums + sub * tl.C + c * VEC + 2 * e) = which ? db[j][e] : dw[j][e];
        }
        __syncthreads();
        for (int c = tid; c < tl.C; c += kBlock) {
            float v = 0.f;
            for (int r = 0; r < kRows; ++r) v += sums[r * tl.C + c];
            p[which * tl.C + c] = v;
        }
    }
}

// dw, db = the blocks' sums added up: 32 columns of part's 2 C by 32 lanes of blocks.
template <typename T>
__global__ void __launch_bounds__(1024)
ln_join_kernel(const float* __restrict__ part, T* __restrict__ dw, T* __restrict__ db, int blocks, int C) {
    __shared__ float s[32][33];
    pdl_enter();  // launched with programmatic dependent launch
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
    float v = 0.f;
    if (c < 2 * C)
        for (int i = ty; i < blocks; i += 32) v += part[(size_t)i * 2 * C + c];
    s[ty][tx] = v;
    __syncthreads();
    v = s[tx][ty];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int col = blockIdx.x * 32 + ty;
    if (tx == 0 && col < 2 * C) {
        if (col < C) {
            if (dw) dw[col] = from_f32<T>(v);
        } else if (db) {
            db[col - C] = from_f32<T>(v);
        }
    }
}

// The row layout for a row of C elements: vectors of 16 bytes where they divide the row, else single elements; as few
// threads for a row as hold it with `most` elements each.
struct Shape {
    bool vec;
    int tpr;
};
Shape row_shape(int C, int elem, int most) {
    Shape r;
    const int V = 16 / elem;
    r.vec = C % V == 0;
    r.tpr = 8;
    while (r.tpr < 1024 && (long long)r.tpr * most < C) r.tpr *= 2;
    return r;
}

constexpr int kFwdElems = 16, kBwdElems = 16;  // elements of a row held by one thread

// Streamed rows: 16-byte vectors divide a row, and in the gradient a row fits on the 256 threads of a block (16
// elements each).  Threads of a row and the tiles' size: about `bytes` to a tile, fewer where there are few rows, a
// multiple of the rows that a block works on at a time.
bool streamed(int C, int elem, bool bwd) { return C % (16 / elem) == 0 && (!bwd || C <= 16 * kBlock); }
int fwd_threads(int C, int elem) {
    const int row = C * elem;
    return row <= 256 ? 8 : row <= 512 ? 16 : row <= 4096 ? 32 : row <= 16384 ? 128 : 256;
}
int bwd_threads(int C) {
    int t = 8;
    while (t * kBwdElems < C) t *= 2;
    return t;
}
Tiles tiles_of(long long rows, int C, int elem, int threads, int bytes) {
    Tiles t{};
    const int at_a_time = kBlock / threads;
    t.rows = rows;
    t.C = C;
    t.row = (uint32_t)C * elem;
    long long r = bytes / (long long)t.row, share = rows / (152 * 4);
    if (r > share) r = share;
    t.R = (int)(r / at_a_time * at_a_time);
    if (t.R < at_a_time) t.R = at_a_time;
    t.tiles = (rows + t.R - 1) / t.R;
    return t;
}
size_t tile_smem(const Tiles& t, int tiles) { return (size_t)tiles * t.row * t.R; }
int resident(size_t smem, int most) {  // blocks of an SM: by shared memory, at most `most` by registers
    const long long per = 225000 / (long long)(smem + 1536);
    return (int)(per < 1 ? 1 : per > most ? most : per);
}
constexpr int kFwdTile = 16384, kBwdTile = 16384;

}  // namespace

int bwd_blocks(const la_norm_shape& s) {
    const int elem = s.dtype == LA_BF16 ? 2 : 4;
    if (streamed(s.C, elem, true)) {
        const Tiles t = tiles_of(s.rows, s.C, elem, bwd_threads(s.C), kBwdTile);
        const long long most = 152LL * resident(tile_smem(t, 2 * kBwdStages), 2);
        return (int)(t.tiles < most ? t.tiles : most);
    }
    const int tpr = row_shape(s.C, elem, kBwdElems).tpr;
    const int rpb = tpr > 32 ? 1 : kBlock / tpr;
    const long long need = (s.rows + rpb - 1) / rpb;
    const long long most = 152LL * (tpr >= 512 ? 2 : 4);
    return (int)(need < most ? need : most);
}

namespace {
template <typename T, int TPR>
cudaError_t fwd_launch(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, long long rows,
                       int C, float eps, cudaStream_t st) {
    constexpr int kRows = TPR > 32 ? 1 : kBlock / TPR;
    long long blocks = (rows + kRows - 1) / kRows;
    if (blocks > 152LL * 64) blocks = 152LL * 64;
    launch_begin("ln_fwd", st);
    const cudaError_t e =
        launch_pdl(ln_fwd_kernel<T, kFwdElems, TPR>, dim3((unsigned)blocks), dim3(TPR > 32 ? TPR : kBlock), 0,
                   st, (const T*)x, (const T*)w, (const T*)b, (T*)y, mean, rstd, rows, C, eps);
    const cudaError_t e2 = launch_end("ln_fwd", st);
    return e != cudaSuccess ? e : e2;
}

template <typename T, int VEC, int TPR>
cudaError_t bwd_launch(const void* x, const void* w, const float* mean, const float* rstd, const void* dy, void* dx,
                       float* part, long long rows, int C, int blocks, cudaStream_t st) {
    constexpr int kRows = TPR > 32 ? 1 : kBlock / TPR;
    const size_t sm = kRows > 1 && part ? (size_t)kRows * C * 4 : 0;
    launch_begin("ln_bwd", st);
    const cudaError_t e = launch_pdl(ln_bwd_kernel<T, VEC, kBwdElems / VEC, TPR>, dim3(blocks),
                                     dim3(TPR > 32 ? TPR : kBlock), sm, st, (const T*)x, (const T*)w, mean, rstd,
                                     (const T*)dy, (T*)dx, part, rows, C);
    const cudaError_t e2 = launch_end("ln_bwd", st);
    return e != cudaSuccess ? e : e2;
}

#define LN_TPR(LAUNCH)                     \
    switch (sh.tpr) {                      \
        case 8: return LAUNCH(8);          \
        case 16: return LAUNCH(16);        \
        case 32: return LAUNCH(32);        \
        case 64: return LAUNCH(64);        \
        case 128: return LAUNCH(128);      \
        case 256: return LAUNCH(256);      \
        case 512: return LAUNCH(512);      \
        default: return LAUNCH(1024);      \
    }

template <typename K, typename... A>
cudaError_t launch_tiles(const char* name, K kern, long long blocks, size_t smem, cudaStream_t st, A... args) {
    cudaError_t e = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    launch_begin(name, st);
    e = launch_pdl(kern, dim3((unsigned)blocks), dim3(kBlock), smem, st, args...);
    const cudaError_t e2 = launch_end(name, st);
    return e != cudaSuccess ? e : e2;
}

template <typename T>
cudaError_t fwd_t(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, long long rows, int C,
                  float eps, cudaStream_t st) {
    if (!streamed(C, sizeof(T), false)) {
        const Shape sh = row_shape(C, sizeof(T), kFwdElems);
#define LN_ROWS(tpr) (fwd_launch<T, tpr>(x, w, b, y, mean, rstd, rows, C, eps, st))
        LN_TPR(LN_ROWS)
#undef LN_ROWS
    }
    const int threads = fwd_threads(C, sizeof(T));
    const Tiles t = tiles_of(rows, C, sizeof(T), threads, kFwdTile);
    const size_t smem = tile_smem(t, kFwdStages);
    const long long most = 152LL * resident(smem, 4), blocks = t.tiles < most ? t.tiles : most;
    int* err = device_error_word();
#define LN_FWD(tpr)                                                                                              \
    return launch_tiles("ln_fwd", ln_fwd_tiles<T, tpr>, blocks, smem, st, (const T*)x, (const T*)w, (const T*)b, (T*)y, \
                        mean, rstd, t, eps, err)
    switch (threads) {
        case 8: LN_FWD(8);
        case 16: LN_FWD(16);
        case 32: LN_FWD(32);
        case 128: LN_FWD(128);
        default: LN_FWD(256);
    }
#undef LN_FWD
}

template <typename T>
cudaError_t bwd_t(const void* x, const void* w, const float* mean, const float* rstd, const void* dy, void* dx,
                  float* part, const la_norm_shape& s, cudaStream_t st) {
    const long long rows = s.rows;
    const int C = s.C, blocks = bwd_blocks(s);
    constexpr int V = 16 / (int)sizeof(T), VPT = kBwdElems / V;
    if (!streamed(C, sizeof(T), true)) {
        const Shape sh = row_shape(C, sizeof(T), kBwdElems);
        if (sh.vec) {  // more than 4096 elements
            if (sh.tpr == 512) return bwd_launch<T, V, 512>(x, w, mean, rstd, dy, dx, part, rows, C, blocks, st);
            return bwd_launch<T, V, 1024>(x, w, mean, rstd, dy, dx, part, rows, C, blocks, st);
        }
#define LN_ROWS(tpr) (bwd_launch<T, 1, tpr>(x, w, mean, rstd, dy, dx, part, rows, C, blocks, st))
        LN_TPR(LN_ROWS)
#undef LN_ROWS
    }
    const int threads = bwd_threads(C);
    const Tiles t = tiles_of(rows, C, sizeof(T), threads, kBwdTile);
    size_t smem = tile_smem(t, 2 * kBwdStages);
    const size_t sums = (size_t)(kBlock / threads) * C * 4;
    if (smem < sums) smem = sums;
    int* err = device_error_word();
#define LN_BWD(tpr)                                                                                                     \
    return launch_tiles("ln_bwd", ln_bwd_tiles<T, VPT, tpr>, blocks, smem, st, (const T*)x, (const T*)w, mean, rstd, \
                        (const T*)dy, (T*)dx, part, t, err)
    switch (threads) {
        case 8: LN_BWD(8);
        case 16: LN_BWD(16);
        case 32: LN_BWD(32);
        case 64: LN_BWD(64);
        case 128: LN_BWD(128);
        default: LN_BWD(256);
    }
#undef LN_BWD
}
}  // namespace

cudaError_t fwd(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, const la_norm_shape& s,
                float eps, cudaStream_t st) {
    return s.dtype == LA_BF16 ? fwd_t<__nv_bfloat16>(x, w, b, y, mean, rstd, s.rows, s.C, eps, st)
                              : fwd_t<float>(x, w, b, y, mean, rstd, s.rows, s.C, eps, st);
}

cudaError_t bwd(const void* x, const void* w, const float* mean, const float* rstd, const void* dy, void* dx, void* dw,
                void* db, float* part, const la_norm_shape& s, cudaStream_t st) {
    float* p = dw || db ? part : nullptr;
    cudaError_t e = s.dtype == LA_BF16 ? bwd_t<__nv_bfloat16>(x, w, mean, rstd, dy, dx, p, s, st)
                                       : bwd_t<float>(x, w, mean, rstd, dy, dx, p, s, st);
    if (e != cudaSuccess || !p) return e;
    const int blocks = bwd_blocks(s);
    const dim3 grid((2 * s.C + 31) / 32);
    launch_begin("ln_join", st);
    e = s.dtype == LA_BF16 ? launch_pdl(ln_join_kernel<__nv_bfloat16>, grid, dim3(1024), 0, st, (const float*)p,
                                        (__nv_bfloat16*)dw, (__nv_bfloat16*)db, blocks, s.C)
                           : launch_pdl(ln_join_kernel<float>, grid, dim3(1024), 0, st, (const float*)p, (float*)dw,
                                        (float*)db, blocks, s.C);
    const cudaError_t e2 = launch_end("ln_join", st);
    return e != cudaSuccess ? e : e2;
}

}  // namespace ln
}  // namespace la
