// gated_delta.cu -- the gated delta rule in fp32 on the CUDA cores, any head size (formulas in gated_delta.cuh).
//
// Forward: gd_prepare (one block per chunk: gates, t, P) and gd_states (one block per head and slice of value
// columns, which are independent of each other: it walks the chunks with its slice of S in shared memory and
// writes o).  Gradient: gd_prepare, gd_sweeps (the forward recurrence for X and the state entering every chunk and,
// beside it, the adjoint one from the last chunk back, sliced alike: dv, Y and the gradient leaving every chunk) and
// gd_grads (one block per chunk: dq, dk, dg, dbeta).  All arithmetic is fp32; sums of log decays fp64.
// Bound by what shared memory returns to registers and, where there are few heads, by the chain of a chunk's products:
// B=2 H=32 N=2048 128 x 128 takes 0.71 ms forward (its operations 0.30 ms at 128 multiply-adds a clock and SM).
#include "gated_delta.cuh"
#include "shared_memory.cuh"

namespace la {
namespace gd {
namespace {

constexpr int kThreads = 256;  // 16 x 16
constexpr int kW = 16;         // value columns that gd_grads walks at a time
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
__device__ __forceinline__ void load_rows(float* dst, const float* __restrict__ src, int c0, int n, int D) {
    const int lg = 31 - __clz(D);  // D is a power of two
    for (int i = threadIdx.x; i < kC * D; i += kThreads) {
        const int r = i >> lg, d = i & (D - 1);
        dst[r * (D + 1) + d] = r < n ? src[(size_t)(c0 + r) * D + d] : 0.f;
    }
}

// acc[i][j] += sum_(x < K) a(i, x) b(x, j); a and b give this thread's rows and columns.
template <int RT, int CT, typename FA, typename FB>  // CT even or 1
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
            if constexpr (CT % 2 == 0) {
#pragma unroll
                for (int j = 0; j < CT; j += 2) {
                    const float2 z = fma2v(make_float2(av[i], av[i]), make_float2(bv[j], bv[j + 1]),
                                           make_float2(acc[i][j], acc[i][j + 1]));
                    acc[i][j] = z.x;
                    acc[i][j + 1] = z.y;
                }
            } else {
                acc[i][0] = fmaf(av[i], bv[0], acc[i][0]);
            }
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
__global__ void __launch_bounds__(kThreads)
gd_prepare(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ g,
           const float* __restrict__ beta, float* __restrict__ recs, float* __restrict__ ts, float* __restrict__ Ps, int N, int M, int Dk) {
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

// ------------------------------------------------------------------ products of the recurrences
// Tiles in shared memory with rows of a multiple of 4 floats.  A thread forms tiles of kR rows by 4 columns: with 4 rows a
// multiply-add costs two bytes of shared-memory reads, with 2 rows three (single columns of four rows cost five and
// were bound by them).
// z[j] += sum_(x < K) a[(kStep j) lda + x] b[x ldb + 0..3]
template <int kStep, int kR>
__device__ __forceinline__ void mac_rows(F4 (&z)[kR], const float* a, int lda, const float* b, int ldb, int K) {
#pragma unroll 2
    for (int x = 0; x < K; x += 4) {
        float4 av[kR], bv[4];
#pragma unroll
        for (int j = 0; j < kR; ++j) av[j] = ld_f4(a + kStep * j * lda + x);
#pragma unroll
        for (int e = 0; e < 4; ++e) bv[e] = ld_f4(b + (x + e) * ldb);
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            fma4(z[j], av[j].x, bv[0]);
            fma4(z[j], av[j].y, bv[1]);
            fma4(z[j], av[j].z, bv[2]);
            fma4(z[j], av[j].w, bv[3]);
        }
    }
}
// z[j] += sum_(x < K) a[x lda + j] b[x ldb + 0..3]: kR consecutive columns of a as rows
template <int kR>
__device__ __forceinline__ void mac_cols(F4 (&z)[kR], const float* a, int lda, const float* b, int ldb, int K) {
#pragma unroll 4
    for (int x = 0; x < K; ++x) {
        const float4 bv = ld_f4(b + x * ldb);
        if constexpr (kR == 4) {
            const float4 av = ld_f4(a + x * lda);
            fma4(z[0], av.x, bv);
            fma4(z[1], av.y, bv);
            fma4(z[2], av.z, bv);
            fma4(z[3], av.w, bv);
        } else {
            const float2 av = *reinterpret_cast<const float2*>(a + x * lda);
            fma4(z[0], av.x, bv);
            fma4(z[1], av.y, bv);
        }
    }
}
template <int kR>
__device__ __forceinline__ void zero(F4 (&z)[kR]) {
#pragma unroll
    for (int j = 0; j < kR; ++j) z[j].a = z[j].b = make_float2(0.f, 0.f);
}
__device__ __forceinline__ F4 scaled(float m, const F4& z) {
    return {make_float2(m * z.a.x, m * z.a.y), make_float2(m * z.b.x, m * z.b.y)};
}

constexpr int kLc4 = kC + 4;  // row pitch of the 64 x 64 tiles

__device__ __forceinline__ void copy16(float* dst, const float* src, bool take) {  // zeros when not taken
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(take ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// Rows [c0, c0 + n) of a [N][D] matrix into dst, pitch D + 4; the rows past n are 0.
template <int kThr>
__device__ __forceinline__ void copy_rows(float* dst, const float* __restrict__ src, int c0, int n, int D) {
    const int lg = 29 - __clz(D);  // D / 4 is a power of two
    for (int i = threadIdx.x; i < kC << lg; i += kThr) {
        const int r = i >> lg, d = 4 * (i & (D / 4 - 1));
        copy16(dst + r * (D + 4) + d, src + (size_t)(c0 + (r < n ? r : 0)) * D + d, r < n);
    }
}
template <int kThr>
__device__ __forceinline__ void copy_square(float* dst, const float* __restrict__ src) {
    for (int i = threadIdx.x; i < kC * kC / 4; i += kThr) copy16(dst + (i >> 4) * kLc4 + 4 * (i & 15), src + 4 * i, true);
}
template <int kThr>
__device__ __forceinline__ void copy_rec(float* dst, const float* __restrict__ src) {
    for (int i = threadIdx.x; i < kRec / 4; i += kThr) copy16(dst + 4 * i, src + 4 * i, true);
}

// ------------------------------------------------------------------ the recurrence over chunks
// Block (slice, head): value columns [W slice, +W), threads with kR x 4 elements of 64 rows each.  o, Xs / Ss (the gradient's records) and S_out may be null.
// K, which the last product of a chunk reads, has two buffers; Q, t and P of the next chunk are copied while the state moves on.
template <int W, int kR>
__device__ __forceinline__ void
states_block(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v, const float* S0,
          const float* __restrict__ recs, const float* __restrict__ ts, const float* __restrict__ Ps,
          float* __restrict__ o, float* __restrict__ Xs, float* __restrict__ Ss, float* S_out, int N, int M, int Dk,
          int Dv) {
    constexpr int kLw = W + 4, kG = kC / kR, kThr = kG * W / 4;
    extern __shared__ __align__(16) float smem[];
    Carve sm{smem};
    const int ld = Dk + 4;
    float* k2 = sm.take(2 * kC * ld);
    float* rec2 = sm.take(2 * kRec);
    float* qs = sm.take(kC * ld);
    float* tt = sm.take(kC * kLc4);
    float* PP = sm.take(kC * kLc4);
    float* S = sm.take(Dk * kLw);
    float* Rb = sm.take(kC * kLw);  // beta R, then tail u
    float* Ub = sm.take(kC * kLw);  // u
    const int tid = threadIdx.x, rg = tid / (W / 4), c = 4 * (tid % (W / 4));
    const size_t bh = blockIdx.y;
    const int col = blockIdx.x * W + c;
    LA_DCHECK(col + 3 < Dv);
    q += bh * N * Dk;
    k += bh * N * Dk;
    auto copy_k = [&](int m) {
        copy_rows<kThr>(k2 + (m & 1) * kC * ld, k, m * kC, min(kC, N - m * kC), Dk);
        copy_rec<kThr>(rec2 + (m & 1) * kRec, recs + (bh * M + m) * kRec);
    };
    auto copy_rest = [&](int m) {
        copy_square<kThr>(tt, ts + (bh * M + m) * kC * kC);
        if (o) {
            copy_square<kThr>(PP, Ps + (bh * M + m) * kC * kC);
            copy_rows<kThr>(qs, q, m * kC, min(kC, N - m * kC), Dk);
        }
    };
    copy_k(0);
    copy_rest(0);
    copies_commit();
    for (int d = rg; d < Dk; d += kG)
        *reinterpret_cast<float4*>(S + d * kLw + c) =
            S0 ? ld_f4(S0 + (bh * Dk + d) * Dv + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int m = 0; m < M; ++m) {
        const int c0 = m * kC, n = min(kC, N - c0);
        const size_t at = bh * M + m;
        const float *ks = k2 + (m & 1) * kC * ld, *rec = rec2 + (m & 1) * kRec;
        float4 vv[kR];
#pragma unroll
        for (int j = 0; j < kR; ++j)
            vv[j] = rg + kG * j < n ? ld_f4(v + (bh * N + c0 + rg + kG * j) * (size_t)Dv + col)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
        copies_wait<0>();
        __syncthreads();  // the chunk's operands and the state are there; the other K has been read
        if (m + 1 < M) copy_k(m + 1);
        copies_commit();
        if (Ss)
            for (int d = rg; d < Dk; d += kG)
                *reinterpret_cast<float4*>(Ss + (at * Dk + d) * Dv + col) = ld_f4(S + d * kLw + c);
        F4 x[kR], w[kR];
        zero(w);
        mac_rows<kG, kR>(w, ks + rg * ld, ld, S + c, kLw, Dk);
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const int r = rg + kG * j;
            x[j] = scaled(-rec[kGam + r], w[j]);
            x[j].a.x += vv[j].x;
            x[j].a.y += vv[j].y;
            x[j].b.x += vv[j].z;
            x[j].b.y += vv[j].w;
            put4(Rb + r * kLw + c, x[j], rec[kBeta + r]);
        }
        __syncthreads();
        mac_rows<kG, kR>(x, tt + rg * kLc4, kLc4, Rb + c, kLw, kC);
        __syncthreads();  // Rb has been read
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const int r = rg + kG * j;
            if (Xs) put4(Xs + (at * kC + r) * Dv + col, x[j]);
            put4(Ub + r * kLw + c, x[j], rec[kBeta + r]);
            put4(Rb + r * kLw + c, x[j], rec[kTb + r]);
        }
        __syncthreads();
        if (o) {
            zero(w);
            mac_rows<kG, kR>(w, qs + rg * ld, ld, S + c, kLw, Dk);
#pragma unroll
            for (int j = 0; j < kR; ++j) w[j] = scaled(rec[kGam + rg + kG * j], w[j]);
            mac_rows<kG, kR>(w, PP + rg * kLc4, kLc4, Ub + c, kLw, kC);
#pragma unroll
            for (int j = 0; j < kR; ++j) {
                const int r = rg + kG * j;
                if (r < n && LA_DCHECK(c0 + r < N)) put4(o + (bh * N + c0 + r) * (size_t)Dv + col, w[j]);
            }
            __syncthreads();  // the old slice, Q and P have been read
        }
        if (m + 1 < M) copy_rest(m + 1);
        copies_commit();
        const float gc = rec[kGam + kC - 1];
        for (int g = rg; g < Dk / kR; g += kG) {
#pragma unroll
            for (int j = 0; j < kR; ++j) w[j] = scaled(gc, get4(S + (kR * g + j) * kLw + c));
            mac_cols(w, ks + kR * g, ld, Rb + c, kLw, kC);
#pragma unroll
            for (int j = 0; j < kR; ++j) put4(S + (kR * g + j) * kLw + c, w[j]);
        }
    }
    __syncthreads();
    if (S_out)
        for (int d = rg; d < Dk; d += kG)
            *reinterpret_cast<float4*>(S_out + (bh * Dk + d) * Dv + col) = ld_f4(S + d * kLw + c);
}

// ------------------------------------------------------------------ the adjoint recurrence, last chunk first
// As above: K in two buffers, Q copied under the products before its own, t and P under the state's.  dS0 may be dS: a block
// reads its slice before it writes it.
template <int W, int kR>
__device__ __forceinline__ void
reverse_block(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ dout,
           const float* __restrict__ recs, const float* __restrict__ ts, const float* __restrict__ Ps,
           float* __restrict__ dv, float* __restrict__ Ys, float* __restrict__ dSs, const float* dS, float* dS0, int N,
           int M, int Dk, int Dv) {
    constexpr int kLw = W + 4, kG = kC / kR, kThr = kG * W / 4;
    extern __shared__ __align__(16) float smem[];
    Carve sm{smem};
    const int ld = Dk + 4;
    float* k2 = sm.take(2 * kC * ld);
    float* rec2 = sm.take(2 * kRec);
    float* qs = sm.take(kC * ld);
    float* tt = sm.take(kC * kLc4);
    float* PP = sm.take(kC * kLc4);
    float* S = sm.take(Dk * kLw);   // this slice of dS'
    float* Db = sm.take(kC * kLw);  // dO, then gam dO
    float* Ub = sm.take(kC * kLw);  // beta dU, then -gam dR
    const int tid = threadIdx.x, rg = tid / (W / 4), c = 4 * (tid % (W / 4));
    const size_t bh = blockIdx.y;
    const int col = blockIdx.x * W + c;
    LA_DCHECK(col + 3 < Dv);
    q += bh * N * Dk;
    k += bh * N * Dk;
    auto copy_k = [&](int m) {
        copy_rows<kThr>(k2 + (m & 1) * kC * ld, k, m * kC, min(kC, N - m * kC), Dk);
        copy_rec<kThr>(rec2 + (m & 1) * kRec, recs + (bh * M + m) * kRec);
    };
    auto copy_squares = [&](int m) {
        copy_square<kThr>(tt, ts + (bh * M + m) * kC * kC);
        copy_square<kThr>(PP, Ps + (bh * M + m) * kC * kC);
    };
    copy_k(M - 1);
    copy_squares(M - 1);
    copies_commit();
    for (int d = rg; d < Dk; d += kG)
        *reinterpret_cast<float4*>(S + d * kLw + c) =
            dS ? ld_f4(dS + (bh * Dk + d) * Dv + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int m = M - 1; m >= 0; --m) {
        const int c0 = m * kC, n = min(kC, N - c0);
        const size_t at = bh * M + m;
        const float *ks = k2 + (m & 1) * kC * ld, *rec = rec2 + (m & 1) * kRec;
        float4 dd[kR];  // rows kR rg + j, here and below
#pragma unroll
        for (int j = 0; j < kR; ++j)
            dd[j] = kR * rg + j < n ? ld_f4(dout + (bh * N + c0 + kR * rg + j) * (size_t)Dv + col)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
        copies_wait<0>();
        __syncthreads();  // the chunk's operands and the state are there; Q and the other K have been read
        copy_rows<kThr>(qs, q, c0, n, Dk);
        copies_commit();
        if (m > 0) copy_k(m - 1);
        copies_commit();
        for (int d = rg; d < Dk; d += kG)
            *reinterpret_cast<float4*>(dSs + (at * Dk + d) * Dv + col) = ld_f4(S + d * kLw + c);
#pragma unroll
        for (int j = 0; j < kR; ++j) *reinterpret_cast<float4*>(Db + (kR * rg + j) * kLw + c) = dd[j];
        F4 y[kR];
        zero(y);
        mac_rows<1, kR>(y, ks + kR * rg * ld, ld, S + c, kLw, Dk);
#pragma unroll
        for (int j = 0; j < kR; ++j) y[j] = scaled(rec[kTail + kR * rg + j], y[j]);
        __syncthreads();  // dO
        mac_cols(y, PP + kR * rg, kLc4, Db + c, kLw, kC);
#pragma unroll
        for (int j = 0; j < kR; ++j) put4(Ub + (kR * rg + j) * kLw + c, y[j], rec[kBeta + kR * rg + j]);
        __syncthreads();
        mac_cols(y, tt + kR * rg, kLc4, Ub + c, kLw, kC);
        copies_wait<1>();  // Q
        __syncthreads();   // Ub, Db, t and P have been read
        if (m > 0) copy_squares(m - 1);
        copies_commit();
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const int r = kR * rg + j;
            put4(Ys + (at * kC + r) * Dv + col, y[j]);
            if (r < n && LA_DCHECK(c0 + r < N)) put4(dv + (bh * N + c0 + r) * (size_t)Dv + col, y[j], rec[kBeta + r]);
            put4(Ub + r * kLw + c, y[j], rec[kBg + r]);
            put4(Db + r * kLw + c, get4(Db + r * kLw + c), rec[kGam + r]);
        }
        __syncthreads();
        const float gc = rec[kGam + kC - 1];
        for (int g = rg; g < Dk / kR; g += kG) {
            F4 s[kR];
#pragma unroll
            for (int j = 0; j < kR; ++j) s[j] = scaled(gc, get4(S + (kR * g + j) * kLw + c));
            mac_cols(s, qs + kR * g, ld, Db + c, kLw, kC);
            mac_cols(s, ks + kR * g, ld, Ub + c, kLw, kC);
#pragma unroll
            for (int j = 0; j < kR; ++j) put4(S + (kR * g + j) * kLw + c, s[j]);
        }
    }
    __syncthreads();
    if (dS0)
        for (int d = rg; d < Dk; d += kG)
            *reinterpret_cast<float4*>(dS0 + (bh * Dk + d) * Dv + col) = ld_f4(S + d * kLw + c);
}

template <int W, int kR>
__global__ void __launch_bounds__(16 * W / kR)
gd_states(FwdArgs a, const float* __restrict__ recs, const float* __restrict__ ts, const float* __restrict__ Ps, int N,
          int M, int Dk, int Dv) {
    states_block<W, kR>((const float*)a.q, (const float*)a.k, (const float*)a.v, a.S0, recs, ts, Ps, (float*)a.o, nullptr,
                        nullptr, a.S, N, M, Dk, Dv);
}

// The gradient's two recurrences do not depend on each other: one grid, the adjoint one (the longer) first.
template <int W, int kR>
__global__ void __launch_bounds__(16 * W / kR)
gd_sweeps(BwdArgs a, const float* __restrict__ recs, const float* __restrict__ ts, const float* __restrict__ Ps,
          float* __restrict__ X, float* __restrict__ Y, float* __restrict__ S, float* __restrict__ dS, int N, int M, int Dk,
          int Dv) {
    if (blockIdx.z == 0)
        reverse_block<W, kR>((const float*)a.q, (const float*)a.k, (const float*)a.dout, recs, ts, Ps, (float*)a.dv, Y, dS,
                             a.dS, a.dS0, N, M, Dk, Dv);
    else
        states_block<W, kR>((const float*)a.q, (const float*)a.k, (const float*)a.v, a.S0, recs, ts, Ps, nullptr, X, S,
                            nullptr, N, M, Dk, Dv);
}

// ------------------------------------------------------------------ dq, dk, dg, dbeta of one chunk
// part[0..63] += the sum over the 16 lanes that share a row (lanes of a half warp: tx).
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int NK>  // Dk = 16 NK
__global__ void __launch_bounds__(kThreads)
gd_grads(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ g,
         const float* __restrict__ dout, const float* __restrict__ recs, const float* __restrict__ Xs, const float* __restrict__ Ys,
         const float* __restrict__ Ss, const float* __restrict__ dSs, float* __restrict__ dq, float* __restrict__ dk,
         float* __restrict__ dg, float* __restrict__ dbeta, int N, int M, int Dv) {
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
    // a slice's values, loaded while the previous one is worked on where one block fills an SM (B=2 H=32 N=2048 128 x 128:
    // 1.11 -> 1.01 ms; with more blocks the registers cost more than the wait: 0.44 -> 0.49 ms at B=1 H=32 N=4096 64 x 64)
    constexpr bool kAhead = NK == 8;
    float xv[4], yv[4], dov[4], sv[NK], dsv[NK];
    auto fetch = [&](int w0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i, c = w0 + tx;
            xv[i] = Xs[(at * kC + r) * Dv + c];
            yv[i] = Ys[(at * kC + r) * Dv + c];
            dov[i] = r < n ? dout[(bh * N + c0 + r) * (size_t)Dv + c] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int r = ty + 16 * i;
            sv[i] = Ss[(at * Dk + r) * Dv + w0 + tx];
            dsv[i] = dSs[(at * Dk + r) * Dv + w0 + tx];
        }
    };
    if (kAhead) fetch(0);
    for (int w0 = 0; w0 < Dv; w0 += kW) {
        if (!kAhead) fetch(w0);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            const float b = rec[kBeta + r];
            ds[r * kLw + tx] = dov[i];
            us[r * kLw + tx] = b * xv[i];
            rs[r * kLw + tx] = b * yv[i];
            const float s = row_sum(xv[i] * yv[i]);
            if (tx == 0) db[r] += s;
        }
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int r = ty + 16 * i;
            Sa[r * (kSt + 1) + tx] = sv[i];
            Sb[r * (kSt + 1) + tx] = dsv[i];
            kept = fmaf(sv[i], dsv[i], kept);
        }
        if (kAhead && w0 + kW < Dv) fetch(w0 + kW);
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
        if (r >= n || !LA_DCHECK(c0 + r < N)) continue;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            dq[(bh * N + c0 + r) * (size_t)Dk + tx + 16 * j] = qi[i][j];
            dk[(bh * N + c0 + r) * (size_t)Dk + tx + 16 * j] = ki[i][j];
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
            const bool reset = g[pos] < kReset;
            const double d = after + (x ? hi : lo) + tail;
            dg[pos] = reset ? 0.f : (float)d;
            dbeta[pos] = db[i];
        }
    }
}

int f4(int n) { return (n + 3) / 4 * 4; }
size_t smem_prepare(int Dk) { return 4 * (size_t)(2 * f4(kC * (Dk + 1)) + kC * kLd + kRec); }
size_t smem_states(int Dk, int W) {
    return 4 * (size_t)(3 * kC * (Dk + 4) + 2 * kC * kLc4 + Dk * (W + 4) + 2 * kC * (W + 4) + 2 * kRec);
}
size_t smem_grads(int Dk) {
    return 4 * (size_t)(2 * f4(kC * (Dk + 1)) + 2 * f4(kC * kLc) + 3 * f4(kC * kLw) + 2 * f4(Dk * 17) + kRec +
                        16 * kC + 3 * kC + kThreads / 32);
}
static_assert(kW == 16, "the staged state columns of gd_grads are one slice");

#define GD_TRY(x)                              \
    do {                                       \
        const cudaError_t _e = (x);            \
        if (_e != cudaSuccess) return _e;      \
    } while (0)

cudaError_t prepare(const void* q, const void* k, const void* g, const void* beta, const Layout& L, char* ws,
                    const la_shape& s, int M, cudaStream_t st) {
    const size_t sm = smem_prepare(s.Dk);
    GD_TRY(allow_smem(gd_prepare, smem_prepare(kMaxHead)));
    launch_begin("gd_prepare", st);
    gd_prepare<<<dim3(M, s.B * s.H), kThreads, sm, st>>>((const float*)q, (const float*)k, (const float*)g,
                                                         (const float*)beta, (float*)(ws + L.rec), (float*)(ws + L.t),
                                                         (float*)(ws + L.P), s.N, M, s.Dk);
    return launch_end("gd_prepare", st);
}

// Value columns of a slice.  Shared memory leaves room for one block to an SM at Dk = 128.  Measured microseconds of a
// chunk there, forward (adjoint) recurrence: 16 columns 5.6 (10.3) in tiles of 2 rows and 6.8 (11.0) of 4; 32 columns 8.2
// (12.5) and 6.8 (12.0); 64 columns 14.7 (23) and 10.6 (16.7).  16 columns are bound by latency, 64 by shared-memory reads.
int slice(const la_shape& s, bool bwd) {
    static constexpr double fwd_us[] = {5.6, 6.8, 10.6}, rev_us[] = {10.3, 12.0, 16.7};
    int best = 16;
    double least = 1e30;
    for (int i = 0; i < 3 && (16 << i) <= s.Dv; ++i) {
        const long long blocks = (long long)s.B * s.H * (s.Dv / (16 << i));
        const double t = finish(bwd ? blocks : 0, rev_us[i], blocks, fwd_us[i]);
        if (t < least) best = 16 << i, least = t;
    }
    return best;
}

template <int W, int kR>
cudaError_t launch_states(const FwdArgs& a, const la_shape& s, const Layout& L, char* ws, int M, cudaStream_t st) {
    const size_t sm = smem_states(s.Dk, W);
    GD_TRY((allow_smem(gd_states<W, kR>, smem_states(kMaxHead, W))));
    launch_begin("gd_states", st);
    gd_states<W, kR><<<dim3(s.Dv / W, s.B * s.H), 16 * W / kR, sm, st>>>(
        a, (const float*)(ws + L.rec), (const float*)(ws + L.t), (const float*)(ws + L.P), s.N, M, s.Dk, s.Dv);
    return launch_end("gd_states", st);
}

template <int W, int kR>
cudaError_t launch_sweeps(const BwdArgs& a, const la_shape& s, const Layout& L, char* ws, int M, cudaStream_t st) {
    const size_t sm = smem_states(s.Dk, W);
    GD_TRY((allow_smem(gd_sweeps<W, kR>, smem_states(kMaxHead, W))));
    launch_begin("gd_sweeps", st);
    gd_sweeps<W, kR><<<dim3(s.Dv / W, s.B * s.H, 2), 16 * W / kR, sm, st>>>(
        a, (const float*)(ws + L.rec), (const float*)(ws + L.t), (const float*)(ws + L.P), (float*)(ws + L.X),
        (float*)(ws + L.Y), (float*)(ws + L.S), (float*)(ws + L.dS), s.N, M, s.Dk, s.Dv);
    return launch_end("gd_sweeps", st);
}

template <int NK>
cudaError_t launch_grads(const BwdArgs& a, const la_shape& s, const Layout& L, char* ws, int M, cudaStream_t st) {
    const size_t sm = smem_grads(s.Dk);
    GD_TRY(allow_smem(gd_grads<NK>, sm));
    launch_begin("gd_grads", st);
    gd_grads<NK><<<dim3(M, s.B * s.H), kThreads, sm, st>>>(
        (const float*)a.q, (const float*)a.k, (const float*)a.g, (const float*)a.dout, (const float*)(ws + L.rec),
        (const float*)(ws + L.X), (const float*)(ws + L.Y), (const float*)(ws + L.S), (const float*)(ws + L.dS),
        (float*)a.dq, (float*)a.dk, (float*)a.dg, (float*)a.dbeta, s.N, M, s.Dv);
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
    const int dk = tc_ok(s) ? tc_dim(s) : s.Dk, dv = tc_ok(s) ? tc_dim(s) : s.Dv;
    L.t = take((tc_ok(s) && bwd ? 3 : 2) * chunks * kC * kC);
    L.P = L.t + chunks * kC * kC * sizeof(float);
    if (bwd) {
        L.X = take(chunks * kC * dv);
        const size_t half = tc_ok(s) ? 2 : 1;  // the states in bf16
        L.Y = take(chunks * kC * dv);
        L.S = take(chunks * dk * dv / half);
        L.dS = take(chunks * dk * dv / half);
    }
    const int M = (s.N + kC - 1) / kC;
    L.segs = tc_ok(s) ? tc_segments(s, bwd) : 1;
    L.cps = (M + L.segs - 1) / L.segs;
    L.segs = (M + L.cps - 1) / L.cps;  // no empty segment
    if (L.segs > 1) {
        const size_t seg = (size_t)s.B * s.H * L.segs * dk * dv;
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

cudaError_t simt_fwd(const FwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    const int M = (s.N + kC - 1) / kC;
    const Layout L = layout(s, false);
    GD_TRY(prepare(a.q, a.k, a.g, a.beta, L, ws, s, M, st));
    switch (slice(s, false)) {
        case 16: return launch_states<16, 2>(a, s, L, ws, M, st);
        case 32: return launch_states<32, 4>(a, s, L, ws, M, st);
        default: return launch_states<64, 4>(a, s, L, ws, M, st);
    }
}

cudaError_t simt_bwd(const BwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    const int M = (s.N + kC - 1) / kC;
    const Layout L = layout(s, true);
    GD_TRY(prepare(a.q, a.k, a.g, a.beta, L, ws, s, M, st));
    switch (slice(s, true)) {
        case 16: GD_TRY((launch_sweeps<16, 2>(a, s, L, ws, M, st))); break;
        case 32: GD_TRY((launch_sweeps<32, 4>(a, s, L, ws, M, st))); break;
        default: GD_TRY((launch_sweeps<64, 4>(a, s, L, ws, M, st))); break;
    }
    switch (s.Dk) {
        case 16: return launch_grads<1>(a, s, L, ws, M, st);
        case 32: return launch_grads<2>(a, s, L, ws, M, st);
        case 64: return launch_grads<4>(a, s, L, ws, M, st);
        default: return launch_grads<8>(a, s, L, ws, M, st);
    }
}

}  // namespace gd
}  // namespace la
