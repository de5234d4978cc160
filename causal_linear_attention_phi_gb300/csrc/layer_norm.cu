// layer_norm.cu -- layer norm over the last dimension, forward and gradient:
//   y = (x - mean) rstd w + b,   mean = sum x / C,   rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   dx = rstd (d - sum d / C - h sum(d h) / C),  d = dy w,  h = (x - mean) rstd;   dw = sum_rows dy h,  db = sum_rows dy
//
// Bound by memory: each element is read once and written once.  A row stays on chip between its passes, so the variance
// is the mean of squared differences from the mean, not a difference of sums.  Tiles of rows are streamed through shared
// memory, worked on in 16-byte vectors where those divide a row (ln_fwd_tiles, ln_bwd_tiles) and by elements where not
// (ln_fwd_elements, ln_bwd_elements).  The gradient's blocks walk rows and keep dw and db of their columns in registers;
// each block writes its sums once and a second kernel adds the blocks' sums in a fixed order (no atomics: the same
// bits every time).  Statistics and sums are fp32; products and fused multiply-adds are written out, so a call gives
// the same bits with and without the statistics returned.
// Measured on one GB300, of the 6.79 TB/s a copy reaches: forward 131072 x 2048 bf16 178 us (0.89), gradient
// 1048576 x 128 bf16 131 us (0.92), 32768 x 8192 bf16 320 us (0.74: 512 threads to a row, one block to an SM).
#include "layer_norm.cuh"
#include "shared_memory.cuh"

namespace la {
namespace ln {
namespace {

constexpr int kBlock = 256;

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

// ------------------------------------------------------------------ streamed rows
// Rows are contiguous, so a tile of them is one bulk copy.  A block keeps two or three tiles in flight in shared memory, which
// is what it takes to keep the memory busy (about 50 KB an SM); rows held in registers instead, with a barrier between
// load and use, reached 0.74 of the copy rate forward (131072 x 2048 bf16; here 0.89) and 0.68 in the gradient
// (1048576 x 128; here 0.92).  What is left is the drain of the last tiles and the statistics.
constexpr int kFwdStages = 2, kBwdStages = 3;

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

struct Tiles {
    long long rows, tiles;
    int C, R;       // R rows to a tile
    uint32_t row;   // bytes of a row
    uint32_t pitch; // bytes from a tile to the next in shared memory
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
        LA_DCHECK(bytes <= tile && k * tl.R + rows_of(k) <= tl.rows);
        sm100::mbar_arrive_expect_tx(bar + s, bytes);
        sm100::bulk_load(smem + s * tile, reinterpret_cast<const uint8_t*>(x) + k * tile, bytes, bar + s);
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
            if (in && !LA_DCHECK(row < tl.rows)) continue;
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
    if (!ok) sm100::mbar_drain(bar, kFwdStages, issued, err, LA_ERR_TIMEOUT);
}

// The gradient: x and dy tiles; a thread keeps dw and db of its columns (VPT vectors) and, up to 16 elements, w.
// `stages` tiles in flight: 3, or as many as shared memory holds of the widest rows.
template <typename T, int VPT, int TPR>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock)
ln_bwd_tiles(const T* x, const T* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
             const T* dy, T* dx, float* __restrict__ part, Tiles tl, int stages, int* err) {
    using P = Pairs<T>;
    constexpr int VEC = 16 / (int)sizeof(T), kThr = TPR > kBlock ? TPR : kBlock, kRows = kThr / TPR;
    constexpr bool kKeep = VPT * VEC <= 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bar[kBwdStages];
    __shared__ float buf[kRows][4][TPR > 256 ? 16 : 8];
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
        const int s = (int)(i % stages);
        const uint32_t bytes = rows_of(k) * tl.row;
        LA_DCHECK(bytes <= tile && k * tl.R + rows_of(k) <= tl.rows);
        sm100::mbar_arrive_expect_tx(bar + s, 2 * bytes);
        sm100::bulk_load(smem + 2 * s * tile, reinterpret_cast<const uint8_t*>(x) + k * tile, bytes, bar + s);
        sm100::bulk_load(smem + (2 * s + 1) * tile, reinterpret_cast<const uint8_t*>(dy) + k * tile, bytes, bar + s);
    };
    for (int i = 0; i < stages; ++i) load(i);
    float2 wv[kKeep ? VPT : 1][P::n], dw[VPT][P::n], db[VPT][P::n];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int e = 0; e < P::n; ++e) {
            wv[kKeep ? i : 0][e] = both(1.f);
            dw[i][e] = db[i][e] = both(0.f);
        }
        if (kKeep && w && t + TPR * i < nv) P::get(reinterpret_cast<const uint4*>(w) + t + TPR * i, wv[kKeep ? i : 0]);
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
    int s = 0, phase = 0;
    for (long long k = blockIdx.x; k < tl.tiles; k += gridDim.x, ++i) {
        const int n = rows_of(k);
        ok = ok && sm100::mbar_wait(bar + s, phase, err, LA_ERR_TIMEOUT);
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
            LA_DCHECK(row < tl.rows);
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
                if (!kKeep && w) P::get(reinterpret_cast<const uint4*>(w) + c, wv[0]);
#pragma unroll
                for (int e = 0; e < P::n; ++e) {
                    const float2 h = mul2(add2(xv[e], both(-mu)), both(rs)), d = mul2(gv[e], wv[kKeep ? j : 0][e]);
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
                if (!kKeep && w) P::get(reinterpret_cast<const uint4*>(w) + c, wv[0]);
#pragma unroll
                for (int e = 0; e < P::n; ++e) {
                    const float2 h = mul2(add2(xv[e], both(-mu)), both(rs)), d = mul2(gv[e], wv[kKeep ? j : 0][e]);
                    gv[e] = mul2(fma2(h, m1, add2(d, m0)), both(rs));
                }
                P::put(o + 16 * c, gv);
            }
        }
        __syncthreads();  // the tiles have been read
        load(i + stages);
        if (++s == stages) s = 0, phase ^= 1;
    }
    if (!ok) sm100::mbar_drain(bar, stages, issued, err, LA_ERR_TIMEOUT);
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
        for (int c = tid; c < tl.C; c += kThr) {
            float v = 0.f;
            for (int r = 0; r < kRows; ++r) v += sums[r * tl.C + c];
            p[which * tl.C + c] = v;
        }
    }
}

// ------------------------------------------------------------------ rows that 16-byte vectors do not divide
// Streamed alike, element by element.  A tile is the aligned bytes around its rows (so it takes some of the rows beside
// it); of the last one, what a copy of whole 16 bytes leaves is fetched by itself.  131072 x 2047 bf16 takes 269 us
// forward and 496 us for the gradient, bound by the instructions to an element; rows loaded from memory into registers
// took 366 and 827 us element by element, and more as vectors with masked ends (508 and 881).
template <typename T>
struct Spans {
    const Tiles& tl;
    long long total;  // bytes
    __device__ explicit Spans(const Tiles& t) : tl(t), total(t.rows * t.row) {}
    __device__ int rows(long long k) const { return (int)min((long long)tl.R, tl.rows - k * tl.R); }
    __device__ long long start(long long k) const { return k * tl.R * tl.row; }
    __device__ uint32_t lead(long long k) const { return (uint32_t)start(k) & 15u; }
    __device__ uint32_t bytes(long long k) const {  // of the copy, from start - lead on
        const long long from = start(k) - lead(k), to = (start(k) + (long long)rows(k) * tl.row + 15) & ~15LL;
        return (uint32_t)((to < total ? to : total & ~15LL) - from);
    }
    // elements that the copy leaves out, into their place
    __device__ void rest(long long k, uint8_t* tile, const T* x) const {
        const long long at = start(k) - lead(k) + bytes(k), left = (start(k) + (long long)rows(k) * tl.row - at) / (long long)sizeof(T);
        if ((long long)threadIdx.x < left)
            reinterpret_cast<T*>(tile + bytes(k))[threadIdx.x] = x[at / (long long)sizeof(T) + threadIdx.x];
    }
    // the copy stays in the rows and in the tile, and leaves out less than a vector
    __device__ bool inside(long long k) const {
        const long long from = start(k) - lead(k), end = start(k) + (long long)rows(k) * tl.row;
        return from >= 0 && from + bytes(k) <= total && bytes(k) <= tl.pitch && end - from <= tl.pitch &&
               (end <= from + bytes(k) || end - from - bytes(k) < 16);
    }
    __device__ bool whole(long long k) const { return start(k) + (long long)rows(k) * tl.row <= (total & ~15LL); }
};

template <typename T, int VPT, int TPR>  // VPT elements to a thread, always the same columns
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock)
ln_fwd_elements(const T* x, const T* __restrict__ w, const T* __restrict__ b, T* y, float* __restrict__ mean,
                float* __restrict__ rstd, Tiles tl, float eps, int* err) {
    constexpr int kThr = TPR > kBlock ? TPR : kBlock, kRows = kThr / TPR;
    constexpr bool kKeep = VPT <= 16;  // the parameters in registers
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bar[kFwdStages];
    __shared__ float buf[kRows][2][TPR > 256 ? 16 : 8];
    const int tid = threadIdx.x, t = tid % TPR, sub = tid / TPR, C = tl.C;
    const Spans<T> sp(tl);
    if (tid == 0) {
        for (int s = 0; s < kFwdStages; ++s) sm100::mbar_init(bar + s, 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();  // launched with programmatic dependent launch
    bool ok = true;
    long long issued = 0;
    auto load = [&](long long i, int s) {  // the i-th tile of this block
        const long long k = blockIdx.x + i * gridDim.x;
        if (tid != 0 || k >= tl.tiles || !ok) return;
        issued = i + 1;
        LA_DCHECK(sp.inside(k));
        sm100::mbar_arrive_expect_tx(bar + s, sp.bytes(k));
        if (sp.bytes(k))
            sm100::bulk_load(smem + s * tl.pitch, reinterpret_cast<const uint8_t*>(x) + sp.start(k) - sp.lead(k), sp.bytes(k), bar + s);
    };
    for (int i = 0; i < kFwdStages; ++i) load(i, i);
    float wv[kKeep ? VPT : 1], bv[kKeep ? VPT : 1];
    if (kKeep) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            wv[kKeep ? j : 0] = w && t + TPR * j < C ? to_f32(w[t + TPR * j]) : 1.f;
            bv[kKeep ? j : 0] = b && t + TPR * j < C ? to_f32(b[t + TPR * j]) : 0.f;
        }
    }
    const float inv = 1.f / (float)C;
    int turn = 0, s = 0, phase = 0;
    long long i = 0;
    for (long long k = blockIdx.x; k < tl.tiles; k += gridDim.x, ++i) {
        const int n = sp.rows(k);
        uint8_t* tile = smem + s * tl.pitch;
        ok = ok && sm100::mbar_wait(bar + s, phase, err, LA_ERR_TIMEOUT);
        __syncwarp();
        if (!sp.whole(k)) {
            sp.rest(k, tile, x);
            __syncthreads();
        }
        const T* rows = reinterpret_cast<const T*>(tile + sp.lead(k));
        for (int r0 = 0; r0 < n; r0 += kRows) {
            const int r = r0 + sub;
            const bool in = r < n;  // the same for a whole warp where a row has a barrier
            if (TPR > 32 && !in) break;
            const T* xr = rows + (in ? r : 0) * C;
            float v[VPT], a[1] = {0.f};
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (t + TPR * j < C) {
                    v[j] = to_f32(xr[t + TPR * j]);
                    a[0] += v[j];
                }
            group_sum<TPR, 1>(a, buf[sub], sub, t, turn);
            const float mu = __fmul_rn(a[0], inv);
            a[0] = 0.f;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (t + TPR * j < C) {
                    v[j] -= mu;
                    a[0] = fmaf(v[j], v[j], a[0]);
                }
            group_sum<TPR, 1>(a, buf[sub], sub, t, turn);
            const float rs = 1.f / sqrtf(fmaf(a[0], inv, eps));
            const long long row = k * tl.R + r;
            if (in && !LA_DCHECK(row < tl.rows)) continue;
            if (in && t == 0) {
                if (mean) mean[row] = mu;
                if (rstd) rstd[row] = rs;
            }
            if (!in) continue;
            T* yr = y + row * C;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = t + TPR * j;
                if (c >= C) continue;
                if (!kKeep) {
                    wv[0] = w ? to_f32(w[c]) : 1.f;
                    bv[0] = b ? to_f32(b[c]) : 0.f;
                }
                yr[c] = from_f32<T>(fmaf(__fmul_rn(v[j], rs), wv[kKeep ? j : 0], bv[kKeep ? j : 0]));
            }
        }
        __syncthreads();  // the tile has been read
        load(i + kFwdStages, s);
        if (++s == kFwdStages) s = 0, phase ^= 1;
    }
    if (!ok) sm100::mbar_drain(bar, kFwdStages, issued, err, LA_ERR_TIMEOUT);
}

template <typename T, int VPT, int TPR>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock)
ln_bwd_elements(const T* x, const T* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
                const T* dy, T* dx, float* __restrict__ part, Tiles tl, int stages, int* err) {
    constexpr int kThr = TPR > kBlock ? TPR : kBlock, kRows = kThr / TPR;
    constexpr bool kKeep = VPT <= 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bar[kBwdStages];
    __shared__ float buf[kRows][4][TPR > 256 ? 16 : 8];
    const int tid = threadIdx.x, t = tid % TPR, sub = tid / TPR, C = tl.C;
    const Spans<T> sp(tl);
    if (tid == 0) {
        for (int s = 0; s < kBwdStages; ++s) sm100::mbar_init(bar + s, 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();  // launched with programmatic dependent launch
    bool ok = true;
    long long issued = 0;
    auto load = [&](long long i, int s) {
        const long long k = blockIdx.x + i * gridDim.x;
        if (tid != 0 || k >= tl.tiles || !ok) return;
        issued = i + 1;
        const long long from = sp.start(k) - sp.lead(k);
        const uint32_t bytes = sp.bytes(k);
        LA_DCHECK(sp.inside(k));
        sm100::mbar_arrive_expect_tx(bar + s, 2 * bytes);
        if (!bytes) return;
        sm100::bulk_load(smem + 2 * s * tl.pitch, reinterpret_cast<const uint8_t*>(x) + from, bytes, bar + s);
        sm100::bulk_load(smem + (2 * s + 1) * tl.pitch, reinterpret_cast<const uint8_t*>(dy) + from, bytes, bar + s);
    };
    for (int i = 0; i < stages; ++i) load(i, i);
    float wv[kKeep ? VPT : 1], dw[VPT], db[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        dw[j] = db[j] = 0.f;
        if (kKeep) wv[kKeep ? j : 0] = w && t + TPR * j < C ? to_f32(w[t + TPR * j]) : 1.f;
    }
    auto weight = [&](int j) { return kKeep ? wv[kKeep ? j : 0] : w ? to_f32(w[t + TPR * j]) : 1.f; };
    const float inv = 1.f / (float)C;
    int turn = 0, s = 0, phase = 0;
    long long i = 0;
    for (long long k = blockIdx.x; k < tl.tiles; k += gridDim.x, ++i) {
        const int n = sp.rows(k);
        uint8_t* tile = smem + 2 * s * tl.pitch;
        ok = ok && sm100::mbar_wait(bar + s, phase, err, LA_ERR_TIMEOUT);
        __syncwarp();
        if (!sp.whole(k)) {
            sp.rest(k, tile, x);
            sp.rest(k, tile + tl.pitch, dy);
            __syncthreads();
        }
        const T *xs = reinterpret_cast<const T*>(tile + sp.lead(k)), *gs = reinterpret_cast<const T*>(tile + tl.pitch + sp.lead(k));
        for (int r0 = 0; r0 < n; r0 += kRows) {
            const int r = r0 + sub;
            const bool in = r < n;
            if (TPR > 32 && !in) break;
            const long long row = k * tl.R + (in ? r : 0);
            LA_DCHECK(row < tl.rows);
            const T *xr = xs + (in ? r : 0) * C, *gr = gs + (in ? r : 0) * C;
            const float mu = mean[row], rs = rstd[row];
            float a[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = t + TPR * j;
                if (!in || c >= C) continue;
                const float g = to_f32(gr[c]), h = __fmul_rn(to_f32(xr[c]) - mu, rs), d = __fmul_rn(g, weight(j));
                a[0] += d;
                a[1] = fmaf(d, h, a[1]);
                dw[j] = fmaf(g, h, dw[j]);
                db[j] += g;
            }
            group_sum<TPR, 2>(a, buf[sub], sub, t, turn);
            if (!in) continue;
            const float m0 = __fmul_rn(a[0], inv), m1 = __fmul_rn(a[1], inv);
            T* o = dx + row * C;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = t + TPR * j;
                if (c >= C) continue;
                const float h = __fmul_rn(to_f32(xr[c]) - mu, rs), d = __fmul_rn(to_f32(gr[c]), weight(j));
                o[c] = from_f32<T>(__fmul_rn(rs, fmaf(-h, m1, d - m0)));
            }
        }
        __syncthreads();  // the tiles have been read
        load(i + stages, s);
        if (++s == stages) s = 0, phase ^= 1;
    }
    if (!ok) sm100::mbar_drain(bar, stages, issued, err, LA_ERR_TIMEOUT);
    if (!part) return;
    float* sums = reinterpret_cast<float*>(smem);
    float* p = part + (size_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
        float* to = kRows == 1 ? p + which * C : sums + sub * C;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (t + TPR * j < C) to[t + TPR * j] = which ? db[j] : dw[j];
        if (kRows == 1) continue;
        __syncthreads();
        for (int c = tid; c < C; c += kThr) {
            float v = 0.f;
            for (int r = 0; r < kRows; ++r) v += sums[r * C + c];
            p[which * C + c] = v;
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
        } else if (db && LA_DCHECK(col - C < C)) {
            db[col - C] = from_f32<T>(v);
        }
    }
}

constexpr int kElems = 16;  // elements of a row held by one thread, 32 of the gradient's widest rows

bool vectors(int C, int elem) { return C % (16 / elem) == 0; }  // 16-byte vectors divide a row
// Threads of a row.  By elements, a thread has 4 or 8 of a short row (always the same columns, few idle).
int element_threads(int C) {
    int t = 8;
    while (t < 32 && t * 4 < C) t *= 2;
    while (t < 512 && t * kElems < C) t *= 2;
    return t;
}
int fwd_threads(int C, int elem) {
    const int row = C * elem;
    if (!vectors(C, elem)) return element_threads(C);
    return row <= 256 ? 8 : row <= 512 ? 16 : row <= 4096 ? 32 : row <= 16384 ? 128 : 256;
}
int bwd_threads(int C, int elem) {
    if (!vectors(C, elem)) return element_threads(C);
    int t = 8;
    while (t < 512 && t * kElems < C) t *= 2;
    return t;
}
int block_of(int threads) { return threads > kBlock ? threads : kBlock; }
// Threads of a row and the tiles' size: about `bytes` to a tile, fewer where there are few rows, a multiple of the rows
// that a block works on at a time.
Tiles tiles_of(long long rows, int C, int elem, int threads, int bytes) {
    Tiles t{};
    const int at_a_time = block_of(threads) / threads;
    t.rows = rows;
    t.C = C;
    t.row = (uint32_t)C * elem;
    long long r = bytes / (long long)t.row, share = rows / (152 * 4);
    if (r > share) r = share;
    t.R = (int)(r / at_a_time * at_a_time);
    if (t.R < at_a_time) t.R = at_a_time;
    t.tiles = (rows + t.R - 1) / t.R;
    t.pitch = (t.row * t.R + (vectors(C, elem) ? 0u : 30u) + 15u) & ~15u;  // up to 15 bytes at either end
    return t;
}
constexpr size_t kMostSmem = 225000;  // of a block; the rest of an SM's is left to static arrays
int resident(size_t smem, int most) {  // blocks of an SM: by shared memory, at most `most` by registers
    const long long per = (long long)kMostSmem / (long long)(smem + 1536);
    return (int)(per < 1 ? 1 : per > most ? most : per);
}
constexpr int kFwdTile = 16384, kBwdTile = 16384;
int bwd_tile(int C, int elem) { return !vectors(C, elem) && C <= 256 ? kBwdTile / 2 : kBwdTile; }  // four blocks to an SM
int bwd_stages(const Tiles& t) {
    const long long fit = (long long)kMostSmem / (2LL * t.pitch);
    return (int)(fit < kBwdStages ? fit : kBwdStages);
}

}  // namespace

int bwd_blocks(const la_norm_shape& s) {
    const int elem = s.dtype == LA_BF16 ? 2 : 4, threads = bwd_threads(s.C, elem);
    const Tiles t = tiles_of(s.rows, s.C, elem, threads, bwd_tile(s.C, elem));
    const int most_by_registers = threads > 256 ? 1 : !vectors(s.C, elem) && s.C <= 256 ? 4 : 2;
    const long long most = 152LL * resident((size_t)2 * bwd_stages(t) * t.pitch, most_by_registers);
    return (int)(t.tiles < most ? t.tiles : most);
}

namespace {
template <typename K, typename... A>
cudaError_t launch_tiles(const char* name, K kern, long long blocks, int block, size_t smem, cudaStream_t st, A... args) {
    cudaError_t e = allow_smem(kern, kMostSmem);
    if (e != cudaSuccess) return e;
    launch_begin(name, st);
    e = launch_pdl(kern, dim3((unsigned)blocks), dim3(block), smem, st, args...);
    const cudaError_t e2 = launch_end(name, st);
    return e != cudaSuccess ? e : e2;
}

template <typename T>
cudaError_t fwd_t(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, long long rows, int C,
                  float eps, cudaStream_t st) {
    const int threads = fwd_threads(C, sizeof(T));
    const Tiles t = tiles_of(rows, C, sizeof(T), threads, kFwdTile);
    const size_t smem = (size_t)kFwdStages * t.pitch;
    int* err = device_error_word();
    auto go = [&](auto kern, int most) {
        const long long all = 152LL * resident(smem, most), blocks = t.tiles < all ? t.tiles : all;
        return launch_tiles("ln_fwd", kern, blocks, block_of(threads), smem, st, (const T*)x, (const T*)w, (const T*)b, (T*)y,
                            mean, rstd, t, eps, err);
    };
    if (!vectors(C, sizeof(T))) {
        if (C <= 4 * threads) {
            if (threads == 8) return go(ln_fwd_elements<T, 4, 8>, 4);
            if (threads == 16) return go(ln_fwd_elements<T, 4, 16>, 4);
            return go(ln_fwd_elements<T, 4, 32>, 4);
        }
        if (C <= 8 * threads) return go(ln_fwd_elements<T, 8, 32>, 4);
        switch (threads) {
            case 32: return go(ln_fwd_elements<T, kElems, 32>, 3);
            case 64: return go(ln_fwd_elements<T, kElems, 64>, 3);
            case 128: return go(ln_fwd_elements<T, kElems, 128>, 3);
            case 256: return go(ln_fwd_elements<T, kElems, 256>, 3);
            default:
                if (C <= 512 * kElems) return go(ln_fwd_elements<T, kElems, 512>, 1);
                return go(ln_fwd_elements<T, 2 * kElems, 512>, 1);
        }
    }
    switch (threads) {
        case 8: return go(ln_fwd_tiles<T, 8>, 4);
        case 16: return go(ln_fwd_tiles<T, 16>, 4);
        case 32: return go(ln_fwd_tiles<T, 32>, 4);
        case 128: return go(ln_fwd_tiles<T, 128>, 4);
        default: return go(ln_fwd_tiles<T, 256>, 4);
    }
}

template <typename T>
cudaError_t bwd_t(const void* x, const void* w, const float* mean, const float* rstd, const void* dy, void* dx,
                  float* part, const la_norm_shape& s, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const int C = s.C, threads = bwd_threads(C, sizeof(T)), blocks = bwd_blocks(s);
    const Tiles t = tiles_of(s.rows, C, sizeof(T), threads, bwd_tile(C, sizeof(T)));
    const int stages = bwd_stages(t);
    size_t smem = (size_t)2 * stages * t.pitch;
    const size_t sums = (size_t)(block_of(threads) / threads) * C * 4;
    if (smem < sums) smem = sums;
    int* err = device_error_word();
    auto go = [&](auto kern) {
        return launch_tiles("ln_bwd", kern, blocks, block_of(threads), smem, st, (const T*)x, (const T*)w, mean, rstd,
                            (const T*)dy, (T*)dx, part, t, stages, err);
    };
    if (!vectors(C, sizeof(T))) {
        if (C <= 4 * threads) {
            if (threads == 8) return go(ln_bwd_elements<T, 4, 8>);
            if (threads == 16) return go(ln_bwd_elements<T, 4, 16>);
            return go(ln_bwd_elements<T, 4, 32>);
        }
        if (C <= 8 * threads) return go(ln_bwd_elements<T, 8, 32>);
        switch (threads) {
            case 32: return go(ln_bwd_elements<T, kElems, 32>);
            case 64: return go(ln_bwd_elements<T, kElems, 64>);
            case 128: return go(ln_bwd_elements<T, kElems, 128>);
            case 256: return go(ln_bwd_elements<T, kElems, 256>);
            default:
                if (C <= 512 * kElems) return go(ln_bwd_elements<T, kElems, 512>);
                return go(ln_bwd_elements<T, 2 * kElems, 512>);
        }
    }
    switch (threads) {
        case 8: return go(ln_bwd_tiles<T, kElems / V, 8>);
        case 16: return go(ln_bwd_tiles<T, kElems / V, 16>);
        case 32: return go(ln_bwd_tiles<T, kElems / V, 32>);
        case 64: return go(ln_bwd_tiles<T, kElems / V, 64>);
        case 128: return go(ln_bwd_tiles<T, kElems / V, 128>);
        case 256: return go(ln_bwd_tiles<T, kElems / V, 256>);
        default:
            if (C <= 512 * kElems) return go(ln_bwd_tiles<T, kElems / V, 512>);
            return go(ln_bwd_tiles<T, 2 * kElems / V, 512>);
    }
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
