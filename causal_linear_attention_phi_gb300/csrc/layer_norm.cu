// layer_norm.cu -- layer norm over the last dimension, forward and gradient:
//   y = (x - mean) rstd w + b,   mean = sum x / C,   rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   dx = rstd (d - sum d / C - h sum(d h) / C),  d = dy w,  h = (x - mean) rstd;   dw = sum_rows dy h,  db = sum_rows dy
//
// Bound by memory: each element is read once and written once.  A row is held in the registers of TPR threads (VPT
// vectors of VEC elements each, 16 bytes where the row length allows it), so the variance is the mean of squared
// differences from the mean, not a difference of sums.  The gradient's blocks walk rows and keep dw
// and db of their columns in registers; each block writes its sums once and a second kernel adds the blocks' sums in
// a fixed order (no atomics: the same bits every time).  Statistics and sums are fp32; products and fused
// multiply-adds are written out, so a call gives the same bits with and without the statistics returned.
#include "la_internal.cuh"
#include "layer_norm.cuh"

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

template <typename T, int VEC, int VPT, int TPR>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock)
ln_fwd_kernel(const T* x, const T* __restrict__ w, const T* __restrict__ b, T* y,
              float* __restrict__ mean, float* __restrict__ rstd, long long rows, int C, float eps) {
    using V = Vec<T, VEC>;
    __shared__ float buf[2][32];
    pdl_enter();  // launched with programmatic dependent launch
    constexpr int kRows = TPR > 32 ? 1 : kBlock / TPR;  // rows of a block
    const int t = threadIdx.x % TPR, sub = TPR > 32 ? 0 : threadIdx.x / TPR, nv = C / VEC;
    const float inv = 1.f / (float)C;
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * kRows; r0 < rows; r0 += (long long)gridDim.x * kRows) {
        const long long r = r0 + sub;
        const bool in = r < rows;
        const V* xr = reinterpret_cast<const V*>(x + r * C);
        V xv[VPT];
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && t + TPR * i < nv) xv[i] = xr[t + TPR * i];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && t + TPR * i < nv)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[0] += to_f32(xv[i].e[e]);
        row_sum<TPR, 1>(s, buf, turn);
        const float mu = __fmul_rn(s[0], inv);
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && t + TPR * i < nv)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = to_f32(xv[i].e[e]) - mu;
                    s[0] = fmaf(d, d, s[0]);
                }
        row_sum<TPR, 1>(s, buf, turn);
        const float rs = 1.f / sqrtf(fmaf(s[0], inv, eps));
        if (in && t == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
        V* yr = reinterpret_cast<V*>(y + r * C);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = t + TPR * i;
            if (!in || c >= nv) continue;
            V wv, bv, o;
            if (w) wv = reinterpret_cast<const V*>(w)[c];
            if (b) bv = reinterpret_cast<const V*>(b)[c];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float h = __fmul_rn(to_f32(xv[i].e[e]) - mu, rs);
                o.e[e] = from_f32<T>(fmaf(h, w ? to_f32(wv.e[e]) : 1.f, b ? to_f32(bv.e[e]) : 0.f));
            }
            yr[c] = o;
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

}  // namespace

int bwd_blocks(long long rows, int C) {
    const int tpr = row_shape(C, 4, kBwdElems).tpr;  // the same for every dtype
    const int rpb = tpr > 32 ? 1 : kBlock / tpr;
    const long long need = (rows + rpb - 1) / rpb;
    const long long most = 152LL * (tpr >= 512 ? 2 : 4);
    return (int)(need < most ? need : most);
}

namespace {
template <typename T, int VEC, int TPR>
cudaError_t fwd_launch(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, long long rows,
                       int C, float eps, cudaStream_t st) {
    constexpr int kRows = TPR > 32 ? 1 : kBlock / TPR;
    long long blocks = (rows + kRows - 1) / kRows;
    if (blocks > 152LL * 64) blocks = 152LL * 64;
    launch_begin("ln_fwd", st);
    const cudaError_t e =
        launch_pdl(ln_fwd_kernel<T, VEC, kFwdElems / VEC, TPR>, dim3((unsigned)blocks), dim3(TPR > 32 ? TPR : kBlock), 0,
                   st, (const T*)x, (const T*)w, (const T*)b, (T*)y, mean, rstd, rows, C, eps);
    const cudaError_t e2 = launch_end("ln_fwd", st);
    return e != cudaSuccess ? e : e2;
}

template <typename T, int VEC, int TPR>
cudaError_t bwd_launch(const void* x, const void* w, const float* mean, const float* rstd, const void* dy, void* dx,
                       float* part, long long rows, int C, cudaStream_t st) {
    constexpr int kRows = TPR > 32 ? 1 : kBlock / TPR;
    const size_t sm = kRows > 1 && part ? (size_t)kRows * C * 4 : 0;
    launch_begin("ln_bwd", st);
    const cudaError_t e = launch_pdl(ln_bwd_kernel<T, VEC, kBwdElems / VEC, TPR>, dim3(bwd_blocks(rows, C)),
                                     dim3(TPR > 32 ? TPR : kBlock), sm, st, (const T*)x, (const T*)w, mean, rstd,
                                     (const T*)dy, (T*)dx, part, rows, C);
    const cudaError_t e2 = launch_end("ln_bwd", st);
    return e != cudaSuccess ? e : e2;
}

#define LN_TPR(fn, VEC, ...)                                      \
    switch (sh.tpr) {                                             \
        case 8: return fn<T, VEC, 8>(__VA_ARGS__);                \
        case 16: return fn<T, VEC, 16>(__VA_ARGS__);              \
        case 32: return fn<T, VEC, 32>(__VA_ARGS__);              \
        case 64: return fn<T, VEC, 64>(__VA_ARGS__);              \
        case 128: return fn<T, VEC, 128>(__VA_ARGS__);            \
        case 256: return fn<T, VEC, 256>(__VA_ARGS__);            \
        case 512: return fn<T, VEC, 512>(__VA_ARGS__);            \
        default: return fn<T, VEC, 1024>(__VA_ARGS__);            \
    }

template <typename T>
cudaError_t fwd_t(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, long long rows, int C,
                  float eps, cudaStream_t st) {
    const Shape sh = row_shape(C, sizeof(T), kFwdElems);
    constexpr int V = 16 / sizeof(T);
    if (sh.vec) LN_TPR(fwd_launch, V, x, w, b, y, mean, rstd, rows, C, eps, st)
    LN_TPR(fwd_launch, 1, x, w, b, y, mean, rstd, rows, C, eps, st)
}

template <typename T>
cudaError_t bwd_t(const void* x, const void* w, const float* mean, const float* rstd, const void* dy, void* dx,
                  float* part, long long rows, int C, cudaStream_t st) {
    const Shape sh = row_shape(C, sizeof(T), kBwdElems);
    constexpr int V = 16 / sizeof(T);
    if (sh.vec) LN_TPR(bwd_launch, V, x, w, mean, rstd, dy, dx, part, rows, C, st)
    LN_TPR(bwd_launch, 1, x, w, mean, rstd, dy, dx, part, rows, C, st)
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
    cudaError_t e = s.dtype == LA_BF16 ? bwd_t<__nv_bfloat16>(x, w, mean, rstd, dy, dx, p, s.rows, s.C, st)
                                       : bwd_t<float>(x, w, mean, rstd, dy, dx, p, s.rows, s.C, st);
    if (e != cudaSuccess || !p) return e;
    const int blocks = bwd_blocks(s.rows, s.C);
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
