// gated_delta.cu -- the gated delta rule on the CUDA cores, any dtype and head size (formulas in gated_delta.cuh).
//
// Forward: gd_prepare (one block per chunk: gates, t, P) and gd_states (one block per head and slice of kW value
// columns, which are independent of each other: it walks the chunks with its slice of S in shared memory and
// writes o).  Gradient: gd_prepare, gd_states (X and the state entering every chunk), gd_reverse (the
// adjoint recurrence from the last chunk back, sliced alike: dv, Y and the gradient leaving every chunk) and
// gd_grads (one block per chunk: dq, dk, dg, dbeta).  All arithmetic is fp32; sums of log decays fp64.
#include "gated_delta.cuh"

namespace la {
namespace gd {
namespace {

constexpr int kThreads = 256;  // 16 x 16
constexpr int kW = 16;         // value columns of a slice
constexpr int kLc = kC + 1;    // row pitch of 64 x 64 tiles
constexpr int kLw = kW + 1;

struct Carve {
    float* p;
    __device__ float* take(int n) {
        float* r = p;
        p += (n + 3) / 4 * 4;
        return r;
    }
};

// Rows [c0, c0 + n) of a [N][D] matrix as fp32 into dst[kC][D + 1]; the rows past n are 0.
template <typename T>
__device__ __forceinline__ void load_rows(float* dst, const T* __restrict__ src, int c0, int n, int D) {
    for (int i = threadIdx.x; i < kC * D; i += kThreads) {
        const int r = i / D, d = i - r * D;
        dst[r * (D + 1) + d] = r < n ? to_f32(src[(size_t)(c0 + r) * D + d]) : 0.f;
    }
}

// acc[i][j] += sum_(x < K) a(i, x) b(x, j); a and b give this thread's rows and columns.
template <int RT, int CT, typename FA, typename FB>
__device__ __forceinline__ void mac(float (&acc)[RT][CT], int K, FA a, FB b) {
#pragma unroll 4
    for (int x = 0; x < K; ++x) {
        float av[RT], bv[CT];
#pragma unroll
        for (int i = 0; i < RT; ++i) av[i] = a(i, x);
#pragma unroll
        for (int j = 0; j < CT; ++j) bv[j] = b(x, j);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
}
template <int RT, int CT>
__device__ __forceinline__ void zero(float (&acc)[RT][CT]) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) acc[i][j] = 0.f;
}

// ------------------------------------------------------------------ gates, t and P of every chunk
template <typename T>
__global__ void __launch_bounds__(kThreads)
gd_prepare(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ g, const T* __restrict__ beta,
           float* __restrict__ recs, float* __restrict__ ts, float* __restrict__ Ps, int N, int M, int Dk) {
    extern __shared__ __align__(16) float smem[];
    Carve sm{smem};
    float* ks = sm.take(kC * (Dk + 1));
    float* qs = sm.take(kC * (Dk + 1));
    float* As = sm.take(kC * kLd);
    float* rec = sm.take(kRec);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, m = blockIdx.x;
    const size_t bh = blockIdx.y;
    const int c0 = m * kC, n = min(kC, N - c0);
    LA_DCHECK(n >= 1 && m < M);
    load_rows(ks, k + bh * N * Dk, c0, n, Dk);
    load_rows(qs, q + bh * N * Dk, c0, n, Dk);
    if (tid < 32) gate_record(g + bh * N, beta + bh * N, c0, n, rec, tid);
    __syncthreads();
    float kk[4][4], qk[4][4];
    zero(kk);
    zero(qk);
    auto col = [&](int x, int j) { return ks[(tx + 16 * j) * (Dk + 1) + x]; };
    mac(kk, Dk, [&](int i, int x) { return ks[(ty + 16 * i) * (Dk + 1) + x]; }, col);
    mac(qk, Dk, [&](int i, int x) { return qs[(ty + 16 * i) * (Dk + 1) + x]; }, col);
    const size_t at = bh * M + m;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = ty + 16 * i, c = tx + 16 * j;
            const float d = r >= c ? pair_decay(rec, r, c) : 0.f;
            // a row that no decay reaches stays 0 whatever the product holds
            As[r * kLd + c] = r > c && d != 0.f ? kk[i][j] * d : 0.f;
            Ps[at * kC * kC + r * kC + c] = d != 0.f ? qk[i][j] * d : 0.f;
        }
    __syncthreads();
    if (tid < 64) solve_diagonal(As, rec + kBeta, tid >> 5, tid & 31);
    __syncthreads();
    solve_joins(As, rec + kBeta, tid);
    for (int i = tid; i < kC * kC; i += kThreads) ts[at * kC * kC + i] = As[(i >> 6) * kLd + (i & 63)];
    for (int i = tid; i < kRec; i += kThreads) recs[at * kRec + i] = rec[i];
}

__device__ __forceinline__ void load_square(float* dst, const float* __restrict__ src) {
    for (int i = threadIdx.x; i < kC * kC; i += kThreads) dst[(i >> 6) * kLc + (i & 63)] = src[i];
}

// ------------------------------------------------------------------ the recurrence over chunks
// Block (slice, head): value columns [kW slice, +kW).  o, Xs / Ss (the gradient's records) and S_out may be null.
template <typename T, int NK>  // Dk = 16 NK
__global__ void __launch_bounds__(kThreads)
gd_states(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const float* __restrict__ S0,
          const float* __restrict__ recs, const float* __restrict__ ts, const float* __restrict__ Ps,
          T* __restrict__ o, float* __restrict__ Xs, float* __restrict__ Ss, float* S_out, int N, int M, int Dv) {
    constexpr int Dk = 16 * NK;
    extern __shared__ __align__(16) float smem[];
    Carve sm{smem};
    float* ks = sm.take(kC * (Dk + 1));
    float* qs = sm.take(kC * (Dk + 1));
    float* tt = sm.take(kC * kLc);
    float* PP = sm.take(kC * kLc);
    float* S = sm.take(Dk * kLw);
    float* Rb = sm.take(kC * kLw);  // beta R, then u = beta X
    float* Ub = sm.take(kC * kLw);
    float* rec = sm.take(kRec);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const size_t bh = blockIdx.y;
    const int col = blockIdx.x * kW + tx;
    LA_DCHECK(col < Dv);
    float s[NK][1];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        s[i][0] = S0 ? S0[(bh * Dk + ty + 16 * i) * Dv + col] : 0.f;
        S[(ty + 16 * i) * kLw + tx] = s[i][0];
    }
    for (int m = 0; m < M; ++m) {
        const int c0 = m * kC, n = min(kC, N - c0);
        const size_t at = bh * M + m;
        __syncthreads();
        load_rows(ks, k + bh * N * Dk, c0, n, Dk);
        load_square(tt, ts + at * kC * kC);
        for (int i = tid; i < kRec; i += kThreads) rec[i] = recs[at * kRec + i];
        if (o) {
            load_rows(qs, q + bh * N * Dk, c0, n, Dk);
            load_square(PP, Ps + at * kC * kC);
        }
        if (Ss) {
#pragma unroll
            for (int i = 0; i < NK; ++i) Ss[(at * Dk + ty + 16 * i) * Dv + col] = s[i][0];
        }
        __syncthreads();
        float x[4][1], w[4][1];
        zero(w);
        mac(w, Dk, [&](int i, int d) { return ks[(ty + 16 * i) * (Dk + 1) + d]; },
            [&](int d, int) { return S[d * kLw + tx]; });
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            const float vv = r < n ? to_f32(v[(bh * N + c0 + r) * (size_t)Dv + col]) : 0.f;
            x[i][0] = fmaf(-rec[kGam + r], w[i][0], vv);
            Rb[r * kLw + tx] = rec[kBeta + r] * x[i][0];
        }
        __syncthreads();
        mac(x, kC, [&](int i, int j) { return tt[(ty + 16 * i) * kLc + j]; },
            [&](int j, int) { return Rb[j * kLw + tx]; });
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            if (Xs) Xs[(at * kC + r) * Dv + col] = x[i][0];
            Ub[r * kLw + tx] = rec[kBeta + r] * x[i][0];
        }
        __syncthreads();
        if (o) {
            zero(w);
            mac(w, Dk, [&](int i, int d) { return qs[(ty + 16 * i) * (Dk + 1) + d]; },
                [&](int d, int) { return S[d * kLw + tx]; });
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i][0] *= rec[kGam + ty + 16 * i];
            mac(w, kC, [&](int i, int j) { return PP[(ty + 16 * i) * kLc + j]; },
                [&](int j, int) { return Ub[j * kLw + tx]; });
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ty + 16 * i;
                if (r < n) o[(bh * N + c0 + r) * (size_t)Dv + col] = from_f32<T>(w[i][0]);
            }
        }
        const float gc = rec[kGam + kC - 1];
#pragma unroll
        for (int i = 0; i < NK; ++i) s[i][0] *= gc;
        mac(s, kC, [&](int i, int j) { return ks[j * (Dk + 1) + ty + 16 * i]; },
            [&](int j, int) { return rec[kTail + j] * Ub[j * kLw + tx]; });
        __syncthreads();  // the old slice has been read
#pragma unroll
        for (int i = 0; i < NK; ++i) S[(ty + 16 * i) * kLw + tx] = s[i][0];
    }
    if (S_out) {
#pragma unroll
        for (int i = 0; i < NK; ++i) S_out[(bh * Dk + ty + 16 * i) * Dv + col] = s[i][0];
    }
}

// ------------------------------------------------------------------ the adjoint recurrence, last chunk first
template <typename T, int NK>
__global__ void __launch_bounds__(kThreads)
gd_reverse(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ dout,
           const float* __restrict__ recs, const float* __restrict__ ts, const float* __restrict__ Ps,
           T* __restrict__ dv, float* __restrict__ Ys, float* __restrict__ dSs, int N, int M, int Dv) {
    constexpr int Dk = 16 * NK;
    extern __shared__ __align__(16) float smem[];
    Carve sm{smem};
    float* ks = sm.take(kC * (Dk + 1));
    float* qs = sm.take(kC * (Dk + 1));
    float* tt = sm.take(kC * kLc);
    float* PP = sm.take(kC * kLc);
    float* S = sm.take(Dk * kLw);   // this slice of dS'
    float* Db = sm.take(kC * kLw);  // dO
    float* Ub = sm.take(kC * kLw);  // beta dU, then -gam dR
    float* rec = sm.take(kRec);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const size_t bh = blockIdx.y;
    const int col = blockIdx.x * kW + tx;
    LA_DCHECK(col < Dv);
    float s[NK][1];
    zero(s);
#pragma unroll
    for (int i = 0; i < NK; ++i) S[(ty + 16 * i) * kLw + tx] = 0.f;
    for (int m = M - 1; m >= 0; --m) {
        const int c0 = m * kC, n = min(kC, N - c0);
        const size_t at = bh * M + m;
        __syncthreads();
        load_rows(ks, k + bh * N * Dk, c0, n, Dk);
        load_rows(qs, q + bh * N * Dk, c0, n, Dk);
        load_square(tt, ts + at * kC * kC);
        load_square(PP, Ps + at * kC * kC);
        for (int i = tid; i < kRec; i += kThreads) rec[i] = recs[at * kRec + i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            Db[r * kLw + tx] = r < n ? to_f32(dout[(bh * N + c0 + r) * (size_t)Dv + col]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NK; ++i) dSs[(at * Dk + ty + 16 * i) * Dv + col] = s[i][0];
        __syncthreads();
        float y[4][1];
        zero(y);
        mac(y, Dk, [&](int i, int d) { return ks[(ty + 16 * i) * (Dk + 1) + d]; },
            [&](int d, int) { return S[d * kLw + tx]; });
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i][0] *= rec[kTail + ty + 16 * i];
        mac(y, kC, [&](int i, int j) { return PP[j * kLc + ty + 16 * i]; },
            [&](int j, int) { return Db[j * kLw + tx]; });
#pragma unroll
        for (int i = 0; i < 4; ++i) Ub[(ty + 16 * i) * kLw + tx] = rec[kBeta + ty + 16 * i] * y[i][0];
        __syncthreads();
        mac(y, kC, [&](int i, int j) { return tt[j * kLc + ty + 16 * i]; },
            [&](int j, int) { return Ub[j * kLw + tx]; });
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            const float dr = rec[kBeta + r] * y[i][0];
            Ys[(at * kC + r) * Dv + col] = y[i][0];
            if (r < n) dv[(bh * N + c0 + r) * (size_t)Dv + col] = from_f32<T>(dr);
            Ub[r * kLw + tx] = -rec[kGam + r] * dr;
            Db[r * kLw + tx] *= rec[kGam + r];
        }
        __syncthreads();
        const float gc = rec[kGam + kC - 1];
#pragma unroll
        for (int i = 0; i < NK; ++i) s[i][0] *= gc;
        mac(s, kC, [&](int i, int j) { return qs[j * (Dk + 1) + ty + 16 * i]; },
            [&](int j, int) { return Db[j * kLw + tx]; });
        mac(s, kC, [&](int i, int j) { return ks[j * (Dk + 1) + ty + 16 * i]; },
            [&](int j, int) { return Ub[j * kLw + tx]; });
#pragma unroll
        for (int i = 0; i < NK; ++i) S[(ty + 16 * i) * kLw + tx] = s[i][0];
    }
}

// ------------------------------------------------------------------ dq, dk, dg, dbeta of one chunk
// part[0..63] += the sum over the 16 lanes that share a row (lanes of a half warp: tx).
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, int NK>
__global__ void __launch_bounds__(kThreads)
gd_grads(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ g, const T* __restrict__ dout,
         const float* __restrict__ recs, const float* __restrict__ Xs, const float* __restrict__ Ys,
         const float* __restrict__ Ss, const float* __restrict__ dSs, T* __restrict__ dq, T* __restrict__ dk,
         T* __restrict__ dg, T* __restrict__ dbeta, int N, int M, int Dv) {
    constexpr int Dk = 16 * NK;
    constexpr int kSt = 16;  // state columns staged at a time
    extern __shared__ __align__(16) float smem[];
    Carve sm{smem};
    float* ks = sm.take(kC * (Dk + 1));
    float* qs = sm.take(kC * (Dk + 1));
    float* Fs = sm.take(kC * kLc);
    float* Es = sm.take(kC * kLc);
    float* ds = sm.take(kC * kLw);  // a slice of dO, u, dR and of S, dS'
    float* us = sm.take(kC * kLw);
    float* rs = sm.take(kC * kLw);
    float* Sa = sm.take(Dk * (kSt + 1));
    float* Sb = sm.take(Dk * (kSt + 1));
    float* rec = sm.take(kRec);
    float* colp = sm.take(16 * kC);  // column sums of the pair products, one row per ty
    float* dG = sm.take(kC);
    float* db = sm.take(kC);
    float* outp = sm.take(kC);
    float* keptp = sm.take(kThreads / 32);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, m = blockIdx.x;
    const size_t bh = blockIdx.y, at = bh * M + m;
    const int c0 = m * kC, n = min(kC, N - c0);
    LA_DCHECK(n >= 1 && m < M);
    load_rows(ks, k + bh * N * Dk, c0, n, Dk);
    load_rows(qs, q + bh * N * Dk, c0, n, Dk);
    for (int i = tid; i < kRec; i += kThreads) rec[i] = recs[at * kRec + i];
    if (tid < kC) db[tid] = 0.f;
    // one walk over the value columns, a slice of kW at a time: dO u^T, dR u^T and the products with the states
    float f[4][4], e[4][4], qi[4][NK], ki[4][NK], ko[4][NK];
    zero(f);
    zero(e);
    zero(qi);
    zero(ki);
    zero(ko);
    float kept = 0.f;
    for (int w0 = 0; w0 < Dv; w0 += kW) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i, c = w0 + tx;
            const float b = rec[kBeta + r];
            const float x = Xs[(at * kC + r) * Dv + c], y = Ys[(at * kC + r) * Dv + c];
            ds[r * kLw + tx] = r < n ? to_f32(dout[(bh * N + c0 + r) * (size_t)Dv + c]) : 0.f;
            us[r * kLw + tx] = b * x;
            rs[r * kLw + tx] = b * y;
            const float s = row_sum(x * y);
            if (tx == 0) db[r] += s;
        }
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int r = ty + 16 * i;
            const float a = Ss[(at * Dk + r) * Dv + w0 + tx], b = dSs[(at * Dk + r) * Dv + w0 + tx];
            Sa[r * (kSt + 1) + tx] = a;
            Sb[r * (kSt + 1) + tx] = b;
            kept = fmaf(a, b, kept);
        }
        __syncthreads();
        auto rowd = [&](int i, int x) { return ds[(ty + 16 * i) * kLw + x]; };
        auto rowr = [&](int i, int x) { return rs[(ty + 16 * i) * kLw + x]; };
        auto rowu = [&](int i, int x) { return us[(ty + 16 * i) * kLw + x]; };
        auto colu = [&](int x, int j) { return us[(tx + 16 * j) * kLw + x]; };
        auto colS = [&](int x, int j) { return Sa[(tx + 16 * j) * (kSt + 1) + x]; };
        auto cold = [&](int x, int j) { return Sb[(tx + 16 * j) * (kSt + 1) + x]; };
        mac(f, kW, rowd, colu);
        mac(e, kW, rowr, colu);
        mac(qi, kW, rowd, colS);
        mac(ki, kW, rowr, colS);
        mac(ko, kW, rowu, cold);
    }
    // F, E and the pair products' share of dG
    {
        float qk[4][4], kk[4][4];
        zero(qk);
        zero(kk);
        auto col = [&](int x, int j) { return ks[(tx + 16 * j) * (Dk + 1) + x]; };
        mac(qk, Dk, [&](int i, int x) { return qs[(ty + 16 * i) * (Dk + 1) + x]; }, col);
        mac(kk, Dk, [&](int i, int x) { return ks[(ty + 16 * i) * (Dk + 1) + x]; }, col);
        float cs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float rsum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty + 16 * i, c = tx + 16 * j;
                const float d = r >= c ? pair_decay(rec, r, c) : 0.f;
                const float F = d != 0.f ? f[i][j] * d : 0.f;
                const float E = d != 0.f && r > c ? -e[i][j] * d : 0.f;
                Fs[r * kLc + c] = F;
                Es[r * kLc + c] = E;
                const float pr = r > c ? fmaf(F, qk[i][j], E * kk[i][j]) : 0.f;
                rsum += pr;
                cs[j] += pr;
            }
            rsum = row_sum(rsum);
            if (tx == 0) dG[ty + 16 * i] = rsum;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) colp[ty * kC + tx + 16 * j] = cs[j];
    }
    // the decays of the products with the states, and their share of dG
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        const float ga = rec[kGam + r], ta = rec[kTail + r];
        float into = 0.f, out = 0.f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int c = tx + 16 * j;
            const float kv = ks[r * (Dk + 1) + c], qv = qs[r * (Dk + 1) + c];
            qi[i][j] *= ga;
            ki[i][j] *= -ga;
            ko[i][j] *= ta;
            into = fmaf(qv, qi[i][j], fmaf(kv, ki[i][j], into));
            out = fmaf(kv, ko[i][j], out);
            ki[i][j] += ko[i][j];
        }
        into = row_sum(into);
        out = row_sum(out);
        if (tx == 0) {
            dG[r] += into - out;
            outp[r] = out;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) kept += __shfl_xor_sync(0xffffffffu, kept, o);
    if ((tid & 31) == 0) keptp[tid >> 5] = kept;
    __syncthreads();
    // dq = qi + F K;  dk = ki + F^T Q + E K + E^T K
    {
        auto kcol = [&](int x, int j) { return ks[x * (Dk + 1) + tx + 16 * j]; };
        auto qcol = [&](int x, int j) { return qs[x * (Dk + 1) + tx + 16 * j]; };
        mac(qi, kC, [&](int i, int x) { return Fs[(ty + 16 * i) * kLc + x]; }, kcol);
        mac(ki, kC, [&](int i, int x) { return Fs[x * kLc + ty + 16 * i]; }, qcol);
        mac(ki, kC, [&](int i, int x) { return Es[(ty + 16 * i) * kLc + x] + Es[x * kLc + ty + 16 * i]; }, kcol);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (r >= n) continue;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            dq[(bh * N + c0 + r) * (size_t)Dk + tx + 16 * j] = from_f32<T>(qi[i][j]);
            dk[(bh * N + c0 + r) * (size_t)Dk + tx + 16 * j] = from_f32<T>(ki[i][j]);
        }
    }
    if (tid < kC) {
        float c = 0.f;
#pragma unroll
        for (int y = 0; y < 16; ++y) c += colp[y * kC + tid];
        dG[tid] -= c;
    }
    __syncthreads();
    if (tid < 32) {  // dg: the reverse cumulative sum, in fp64 (its terms cancel)
        double tail = 0.0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) tail += (double)keptp[w];
        tail *= (double)rec[kGam + kC - 1];
        double os = (double)outp[2 * tid] + (double)outp[2 * tid + 1];
        const double hi = dG[2 * tid + 1], lo = (double)dG[2 * tid] + hi;
        double run = lo;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_down_sync(0xffffffffu, run, o);
            if (tid + o < 32) run += x;
            os += __shfl_xor_sync(0xffffffffu, os, o);
        }
        tail += os;
        const double after = run - lo;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = 2 * tid + x;
            if (i >= n) continue;
            const size_t pos = bh * N + c0 + i;
            const bool reset = to_f32(g[pos]) < kReset;
            const double d = after + (x ? hi : lo) + tail;
            dg[pos] = from_f32<T>(reset ? 0.f : (float)d);
            dbeta[pos] = from_f32<T>(db[i]);
        }
    }
}

int f4(int n) { return (n + 3) / 4 * 4; }
size_t smem_prepare(int Dk) { return 4 * (size_t)(2 * f4(kC * (Dk + 1)) + kC * kLd + kRec); }
size_t smem_states(int Dk) {
    return 4 * (size_t)(2 * f4(kC * (Dk + 1)) + 2 * f4(kC * kLc) + f4(Dk * kLw) + 2 * f4(kC * kLw) + kRec);
}
size_t smem_grads(int Dk) {
    return 4 * (size_t)(2 * f4(kC * (Dk + 1)) + 2 * f4(kC * kLc) + 3 * f4(kC * kLw) + 2 * f4(Dk * 17) + kRec +
                        16 * kC + 3 * kC + kThreads / 32);
}
static_assert(kW == 16, "the staged state columns of gd_grads are one slice");

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
    return cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

#define GD_TRY(x)                              \
    do {                                       \
        const cudaError_t _e = (x);            \
        if (_e != cudaSuccess) return _e;      \
    } while (0)

template <typename T>
cudaError_t prepare(const void* q, const void* k, const void* g, const void* beta, const Layout& L, char* ws,
                    const la_shape& s, int M, cudaStream_t st) {
    const size_t sm = smem_prepare(s.Dk);
    GD_TRY(allow_smem(gd_prepare<T>, sm));
    launch_begin("gd_prepare", st);
    gd_prepare<T><<<dim3(M, s.B * s.H), kThreads, sm, st>>>(
        (const T*)q, (const T*)k, (const T*)g, (const T*)beta, (float*)(ws + L.rec), (float*)(ws + L.t),
        (float*)(ws + L.P), s.N, M, s.Dk);
    return launch_end("gd_prepare", st);
}

template <typename T, int NK>
cudaError_t fwd_t(const FwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    const int M = (s.N + kC - 1) / kC;
    const Layout L = layout(s, false);
    GD_TRY(prepare<T>(a.q, a.k, a.g, a.beta, L, ws, s, M, st));
    const size_t sm = smem_states(s.Dk);
    auto kern = gd_states<T, NK>;
    GD_TRY(allow_smem(kern, sm));
    launch_begin("gd_states", st);
    kern<<<dim3(s.Dv / kW, s.B * s.H), kThreads, sm, st>>>(
        (const T*)a.q, (const T*)a.k, (const T*)a.v, a.S0, (const float*)(ws + L.rec), (const float*)(ws + L.t),
        (const float*)(ws + L.P), (T*)a.o, nullptr, nullptr, a.S, s.N, M, s.Dv);
    return launch_end("gd_states", st);
}

template <typename T, int NK>
cudaError_t bwd_t(const BwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    const int M = (s.N + kC - 1) / kC, BH = s.B * s.H;
    const Layout L = layout(s, true);
    float *rec = (float*)(ws + L.rec), *t = (float*)(ws + L.t), *P = (float*)(ws + L.P);
    float *X = (float*)(ws + L.X), *Y = (float*)(ws + L.Y), *S = (float*)(ws + L.S), *dS = (float*)(ws + L.dS);
    GD_TRY(prepare<T>(a.q, a.k, a.g, a.beta, L, ws, s, M, st));
    const size_t sm = smem_states(s.Dk);
    auto states = gd_states<T, NK>;
    GD_TRY(allow_smem(states, sm));
    launch_begin("gd_states", st);
    states<<<dim3(s.Dv / kW, BH), kThreads, sm, st>>>((const T*)a.q, (const T*)a.k, (const T*)a.v, nullptr, rec, t,
                                                       P, nullptr, X, S, nullptr, s.N, M, s.Dv);
    GD_TRY(launch_end("gd_states", st));
    auto reverse = gd_reverse<T, NK>;
    GD_TRY(allow_smem(reverse, sm));
    launch_begin("gd_reverse", st);
    reverse<<<dim3(s.Dv / kW, BH), kThreads, sm, st>>>((const T*)a.q, (const T*)a.k, (const T*)a.dout, rec, t, P,
                                                        (T*)a.dv, Y, dS, s.N, M, s.Dv);
    GD_TRY(launch_end("gd_reverse", st));
    const size_t smg = smem_grads(s.Dk);
    auto grads = gd_grads<T, NK>;
    GD_TRY(allow_smem(grads, smg));
    launch_begin("gd_grads", st);
    grads<<<dim3(M, BH), kThreads, smg, st>>>((const T*)a.q, (const T*)a.k, (const T*)a.g, (const T*)a.dout, rec, X,
                                              Y, S, dS, (T*)a.dq, (T*)a.dk, (T*)a.dg, (T*)a.dbeta, s.N, M, s.Dv);
    return launch_end("gd_grads", st);
}

}  // namespace

Layout layout(const la_shape& s, bool bwd) {
    Layout L{};
    const size_t chunks = (size_t)s.B * s.H * ((s.N + kC - 1) / kC);
    size_t off = 0;
    auto take = [&](size_t floats) {
        const size_t at = off;
        off += (floats * 4 + 255) / 256 * 256;
        return at;
    };
    L.rec = take(chunks * kRec);
    L.t = take((tc_ok(s) && bwd ? 3 : 2) * chunks * kC * kC);
    L.P = L.t + chunks * kC * kC * sizeof(float);
    if (bwd) {
        L.X = take(chunks * kC * s.Dv);
        const size_t half = tc_ok(s) ? 2 : 1;  // the states in bf16
        L.Y = take(chunks * kC * s.Dv);
        L.S = take(chunks * s.Dk * s.Dv / half);
        L.dS = take(chunks * s.Dk * s.Dv / half);
    }
    const int M = (s.N + kC - 1) / kC;
    L.segs = tc_ok(s) ? tc_segments(s, bwd) : 1;
    L.cps = (M + L.segs - 1) / L.segs;
    L.segs = (M + L.cps - 1) / L.cps;  // no empty segment
    if (L.segs > 1) {
        const size_t seg = (size_t)s.B * s.H * L.segs * s.Dk * s.Dv;
        L.segB = take(seg);
        L.segM = take(seg);
        L.segS = take(seg);
        if (bwd) {
            L.segB2 = take(seg);
            L.segdS = take(seg);
        }
    }
    L.bytes = off;
    return L;
}

#define GD_DISPATCH(fn, ...)                                                             \
    do {                                                                                 \
        if (s.dtype == LA_BF16) {                                                        \
            switch (s.Dk) {                                                              \
                case 16: return fn<__nv_bfloat16, 1>(__VA_ARGS__);                       \
                case 32: return fn<__nv_bfloat16, 2>(__VA_ARGS__);                       \
                case 64: return fn<__nv_bfloat16, 4>(__VA_ARGS__);                       \
                default: return fn<__nv_bfloat16, 8>(__VA_ARGS__);                       \
            }                                                                            \
        }                                                                                \
        switch (s.Dk) {                                                                  \
            case 16: return fn<float, 1>(__VA_ARGS__);                                   \
            case 32: return fn<float, 2>(__VA_ARGS__);                                   \
            case 64: return fn<float, 4>(__VA_ARGS__);                                   \
            default: return fn<float, 8>(__VA_ARGS__);                                   \
        }                                                                                \
    } while (0)

cudaError_t simt_fwd(const FwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    GD_DISPATCH(fwd_t, a, s, ws, st);
}
cudaError_t simt_bwd(const BwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    GD_DISPATCH(bwd_t, a, s, ws, st);
}

}  // namespace gd
}  // namespace la
