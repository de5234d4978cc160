// gated_delta_step.cu -- one position of the gated delta rule for every head, the state updated in place:
//   w = S^T k,  u = beta (v - a w),  S <- a S + k u^T,  out = S^T q = a S_old^T q + (q . k) u,   a = exp(g).
//
// Bound by the state's traffic (fp32, read and written once).  A head's state is held in registers by TPH
// threads as float4s, every load issued before any arithmetic; S^T k and S^T q are formed in the same walk over it,
// so there is one reduction and the state is touched once.
#include "gated_delta.cuh"

namespace la {
namespace gd {
namespace {

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ void st4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void st4(__nv_bfloat16* p, float4 x) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
__device__ __forceinline__ void add4(float4& a, const float4& b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}
__device__ __forceinline__ void fma4(float4& a, float s, const float4& b) {
    a.x = fmaf(s, b.x, a.x);
    a.y = fmaf(s, b.y, a.y);
    a.z = fmaf(s, b.z, a.z);
    a.w = fmaf(s, b.w, a.w);
}
__device__ __forceinline__ void xor4(float4& a, int o) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
}

// Threads for one head: at most 16 float4 of the state each.
template <int DK, int DV>
struct Cfg {
    static constexpr int kF4 = DK * DV / 4;
    static constexpr int kTph = kF4 / 16 < 32 ? 32 : kF4 / 16;
    static constexpr int kHeads = kTph == 32 ? 2 : 1;  // heads of a block
    static constexpr int kCols = DV / 4;               // threads across a row
    static constexpr int kGroups = kTph / kCols;       // rows side by side
    static constexpr int kRows = DK / kGroups;         // rows of a thread: group + kGroups x
    static constexpr int kWarps = kTph / 32;
};

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(Cfg<DK, DV>::kTph* Cfg<DK, DV>::kHeads)
gd_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ g,
               const T* __restrict__ beta, float* __restrict__ S, T* __restrict__ out, int BH) {
    using C = Cfg<DK, DV>;
    __shared__ float qs[C::kHeads][DK], ks[C::kHeads][DK];
    __shared__ float4 part[C::kWarps][2][C::kCols];
    __shared__ float partqk[C::kWarps];
    pdl_enter();  // launched with programmatic dependent launch
    const int sub = threadIdx.x / C::kTph, t = threadIdx.x % C::kTph, lane = threadIdx.x & 31;
    const int h = blockIdx.x * C::kHeads + sub;
    if (h >= BH) return;  // a whole warp (kHeads > 1 only where a head is one warp)
    const int col = t % C::kCols * 4, grp = t / C::kCols;
    LA_DCHECK(col + 3 < DV && grp + C::kGroups * (C::kRows - 1) < DK && sub < C::kHeads);
    float* Sh = S + (size_t)h * (DK * DV);
    float4 s[C::kRows];
#pragma unroll
    for (int x = 0; x < C::kRows; ++x) s[x] = ld4(Sh + (grp + C::kGroups * x) * DV + col);
    for (int d = t; d < DK; d += C::kTph) {
        qs[sub][d] = to_f32(q[(size_t)h * DK + d]);
        ks[sub][d] = to_f32(k[(size_t)h * DK + d]);
    }
    const float4 vv = ld4(v + (size_t)h * DV + col);
    const float a = expf(to_f32(g[h])), b = to_f32(beta[h]);
    if (C::kWarps == 1)
        __syncwarp();
    else
        __syncthreads();
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f), o = w;
    float qk = 0.f;
#pragma unroll
    for (int x = 0; x < C::kRows; ++x) {
        const float kd = ks[sub][grp + C::kGroups * x], qd = qs[sub][grp + C::kGroups * x];
        fma4(w, kd, s[x]);
        fma4(o, qd, s[x]);
        qk = fmaf(qd, kd, qk);
    }
#pragma unroll
    for (int off = C::kCols; off < 32; off <<= 1) {
        xor4(w, off);
        xor4(o, off);
        qk += __shfl_xor_sync(0xffffffffu, qk, off);
    }
    if (C::kWarps > 1) {
        const int warp = t >> 5;
        if (lane < C::kCols) {
            part[warp][0][lane] = w;
            part[warp][1][lane] = o;
        }
        if (lane == 0) partqk[warp] = qk;
        __syncthreads();
        w = o = make_float4(0.f, 0.f, 0.f, 0.f);
        qk = 0.f;
#pragma unroll
        for (int x = 0; x < C::kWarps; ++x) {
            add4(w, part[x][0][col / 4]);
            add4(o, part[x][1][col / 4]);
            qk += partqk[x];
        }
    }
    const float4 u = make_float4(b * fmaf(-a, w.x, vv.x), b * fmaf(-a, w.y, vv.y), b * fmaf(-a, w.z, vv.z),
                                 b * fmaf(-a, w.w, vv.w));
#pragma unroll
    for (int x = 0; x < C::kRows; ++x) {
        const int r = grp + C::kGroups * x;
        float4 n = make_float4(a * s[x].x, a * s[x].y, a * s[x].z, a * s[x].w);
        fma4(n, ks[sub][r], u);
        *reinterpret_cast<float4*>(Sh + r * DV + col) = n;
    }
    if (grp == 0)
        st4(out + (size_t)h * DV + col, make_float4(fmaf(qk, u.x, a * o.x), fmaf(qk, u.y, a * o.y),
                                                    fmaf(qk, u.z, a * o.z), fmaf(qk, u.w, a * o.w)));
}

template <typename T, int DK, int DV>
cudaError_t launch(const void* q, const void* k, const void* v, const void* g, const void* beta, float* S, void* out,
                   int BH, cudaStream_t st) {
    using C = Cfg<DK, DV>;
    launch_begin("gd_step", st);
    const cudaError_t e = launch_pdl(gd_step_kernel<T, DK, DV>, dim3((BH + C::kHeads - 1) / C::kHeads),
                                     dim3(C::kTph * C::kHeads), 0, st, (const T*)q, (const T*)k, (const T*)v,
                                     (const T*)g, (const T*)beta, S, (T*)out, BH);
    const cudaError_t e2 = launch_end("gd_step", st);
    return e != cudaSuccess ? e : e2;
}

template <typename T>
cudaError_t step_t(const void* q, const void* k, const void* v, const void* g, const void* beta, float* S, void* out,
                   const la_shape& s, cudaStream_t st) {
    const int BH = s.B * s.H;
#define GD_STEP(a, b) \
    if (s.Dk == a && s.Dv == b) return launch<T, a, b>(q, k, v, g, beta, S, out, BH, st);
    GD_STEP(16, 16) GD_STEP(16, 32) GD_STEP(16, 64) GD_STEP(16, 128)
    GD_STEP(32, 16) GD_STEP(32, 32) GD_STEP(32, 64) GD_STEP(32, 128)
    GD_STEP(64, 16) GD_STEP(64, 32) GD_STEP(64, 64) GD_STEP(64, 128)
    GD_STEP(128, 16) GD_STEP(128, 32) GD_STEP(128, 64) GD_STEP(128, 128)
#undef GD_STEP
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t step(const void* q, const void* k, const void* v, const void* g, const void* beta, float* S, void* out,
                 const la_shape& s, cudaStream_t st) {
    return s.dtype == LA_BF16 ? step_t<__nv_bfloat16>(q, k, v, g, beta, S, out, s, st)
                              : step_t<float>(q, k, v, g, beta, S, out, s, st);
}

}  // namespace gd
}  // namespace la
