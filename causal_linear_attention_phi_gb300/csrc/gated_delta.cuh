// gated_delta.cuh -- the gated delta rule (itwiki 선형 어텐션, 발전: 감쇠, 게이트, 델타 규칙: a decaying
// state whose write replaces what the key already holds).  Per head, with S a Dk x Dv state:
//   a_t = exp(g_t),  u_t = beta_t (v_t - a_t S_(t-1)^T k_t),  S_t = a_t S_(t-1) + k_t u_t^T,  o_t = S_t^T q_t.
//
// Chunked form, for a chunk of C = 64 positions entered with the state S.  With G_i the sum of g over the
// chunk's positions up to i, gam_i = exp(G_i), tail_j = exp(G_C - G_j), and Gam_ij = exp(G_i - G_j) for i >= j:
//   A = tril(K K^T, -1) . Gam                        what earlier keys of the chunk hold of key i
//   R = V - gam K S,   u = beta X,   X = R - A u     (X is v minus what the state before t holds of k_t)
//     =>  X = R + t (beta R)  with  t = -A (I + beta A)^-1, strictly lower triangular
//   O  = gam Q S + P u,   P = tril(Q K^T) . Gam
//   S' = gam_C S + K^T (tail u)
// Gradient, with dS' the gradient with respect to the state after the chunk:
//   dU = P^T dO + tail K dS',   Y = dU + t^T (beta dU),   dV = dR = beta Y,   dbeta_i = X_i . Y_i
//   dS = gam_C dS' + Q^T (gam dO) - K^T (gam dR)
//   F = tril(dO u^T) . Gam,   E = -tril(dR u^T, -1) . Gam
//   dQ = gam dO S^T + F K
//   dK = tail u dS'^T + F^T Q + E K + E^T K - gam dR S^T
//   dG_i: every product that a decay enters counted at its later end and taken off at its earlier one;
//   dg = the reverse cumulative sum of dG.
// t is kept apart from the identity, so neither beta nor a decay is ever divided by: beta = 0 and
// a = 0 are ordinary values.
#pragma once

#include "la_internal.cuh"

namespace la {
namespace gd {

constexpr int kC = 64;

// The gates of one chunk, fp32, one record per (head, chunk) in the workspace.  The sum of log decays (to the base
// 2 here) is formed in fp64 and kept as hi + lo, so that differences of long sums keep fp32's precision; a decay
// below exp(-100) (under fp32's normal range; -inf among them) is counted in kSeg instead of entering the sum,
// and a product across it is 0.  Positions past the sequence's end have g = 0 and beta = 0.
constexpr int kGam = 0, kNg = kC, kTb = 2 * kC, kTail = 3 * kC, kBeta = 4 * kC, kBg = 5 * kC;  // -gam, tail beta, -beta gam
constexpr int kGhi = 6 * kC, kGlo = 7 * kC, kSeg = 8 * kC;
constexpr int kRec = 9 * kC;
constexpr float kReset = -100.f;

// 2^(hi + lo) for |lo| at most half a step of hi.
__device__ __forceinline__ float exp2_hilo(float hi, float lo) {
    const float e = exp2f(hi);
    return fmaf(e, lo * 0.6931471805599453f, e);
}

// Gam_ij for i >= j (0 across a reset).
__device__ __forceinline__ float pair_decay(const float* rec, int i, int j) {
    return rec[kSeg + i] == rec[kSeg + j]
               ? exp2_hilo(rec[kGhi + i] - rec[kGhi + j], rec[kGlo + i] - rec[kGlo + j])
               : 0.f;
}

// One warp forms the record of the chunk at c0 (n positions) in rec (shared memory).
template <typename T>
__device__ __forceinline__ void gate_record(const T* __restrict__ g, const T* __restrict__ beta, int c0, int n,
                                            float* rec, int lane) {
    double v[2];
    int r[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        const float x = i < n ? to_f32(g[c0 + i]) : 0.f;
        const bool reset = x < kReset;
        v[e] = reset ? 0.0 : (double)x * 1.4426950408889634074;
        r[e] = reset ? 1 : 0;
    }
    v[1] += v[0];
    r[1] += r[0];
    double sv = v[1];
    int sr = r[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double pv = __shfl_up_sync(0xffffffffu, sv, o);
        const int pr = __shfl_up_sync(0xffffffffu, sr, o);
        if (lane >= o) {
            sv += pv;
            sr += pr;
        }
    }
    const double tot = __shfl_sync(0xffffffffu, sv, 31);
    const int rtot = __shfl_sync(0xffffffffu, sr, 31);
    const double base = sv - v[1];
    const int rbase = sr - r[1];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        const double G = base + v[e], D = tot - G;
        const int seg = rbase + r[e];
        const float hi = (float)G, lo = (float)(G - (double)hi);
        const float dhi = (float)D, dlo = (float)(D - (double)dhi);
        rec[kGhi + i] = hi;
        rec[kGlo + i] = lo;
        rec[kSeg + i] = (float)seg;
        const float gam = seg == 0 ? exp2_hilo(hi, lo) : 0.f, tail = seg == rtot ? exp2_hilo(dhi, dlo) : 0.f;
        const float b = i < n ? to_f32(beta[c0 + i]) : 0.f;
        rec[kGam + i] = gam;
        rec[kNg + i] = -gam;
        rec[kTail + i] = tail;
        rec[kBeta + i] = b;
        rec[kBg + i] = -b * gam;
        rec[kTb + i] = tail * b;
    }
}

constexpr int kLd = kC + 4;  // row pitch of A

__device__ __forceinline__ float4 ld_f4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// a += m b on two floats at once.
__device__ __forceinline__ void fma2(float2& a, float m, float2 b) {
    const float2 mm = make_float2(m, m);
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<uint64_t&>(a))
        : "l"(reinterpret_cast<const uint64_t&>(mm)), "l"(reinterpret_cast<const uint64_t&>(b)));
}
// a b + c on two floats at once.
__device__ __forceinline__ float2 fma2v(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
          "l"(reinterpret_cast<const uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2v(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2v(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
    return d;
}
struct F4 {
    float2 a, b;
};
__device__ __forceinline__ void fma4(F4& z, float m, float4 v) {
    fma2(z.a, m, make_float2(v.x, v.y));
    fma2(z.b, m, make_float2(v.z, v.w));
}
__device__ __forceinline__ F4 get4(const float* p) {
    const float4 v = ld_f4(p);
    return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ void put4(float* p, const F4& z, float s = 1.f) {
    *reinterpret_cast<float4*>(p) = make_float4(s * z.a.x, s * z.a.y, s * z.b.x, s * z.b.y);
}
// z[j] += sum_(k0 <= k < k1) row[j step kLd + k] beta[k] m[k][0..3] for the J rows from j0 on, m's rows kLd apart; k0 and
// k1 multiples of 4.  A load from shared memory costs the bytes it returns to registers, broadcast or not (these
// products are bound by that: 4 x 4 tiles return 2.25 bytes a multiply-add, single rows of 8 columns 5).
template <int kJ0, int kStep>
__device__ __forceinline__ void acc_tile(F4 (&z)[4], const float* row, const float* beta, const float* m, int k0, int k1) {
#pragma unroll 2
    for (int k = k0; k < k1; k += 4) {
        const float4 be = ld_f4(beta + k);
        float4 a[4], v[4];
#pragma unroll
        for (int j = kJ0; j < 4; ++j) a[j] = ld_f4(row + j * kStep * kLd + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ld_f4(m + (k + e) * kLd);
#pragma unroll
        for (int j = kJ0; j < 4; ++j) {
            fma4(z[j], a[j].x * be.x, v[0]);
            fma4(z[j], a[j].y * be.y, v[1]);
            fma4(z[j], a[j].z * be.z, v[2]);
            fma4(z[j], a[j].w * be.w, v[3]);
        }
    }
}

// t = -A (I + beta A)^-1 in place of a strictly lower triangular A (zero on and above the diagonal), 64 x 64 fp32 in
// shared memory with row pitch kLd.  Four diagonal blocks of 16 by forward substitution,
// t_i = -(A_i + sum_(j<i) A_ij beta_j t_j), one column to a lane, the column in registers; then blocks are joined in
// pairs, first to 32 and then to 64: t21 = -(I + t22 beta) A21 (I + beta t11), two small products each.  (Diagonal
// blocks of 32 left all but two warps waiting for a chain of 31 rows.)
// solve_diagonal: one warp, the two diagonal blocks of rows 32 w .. 32 w + 31, which it needs complete.  A row is loaded
// while the one before it is solved, and takes the newest value last: a row then waits for one multiply-add.
__device__ __forceinline__ void solve_diagonal(float* A, const float* beta, int w, int lane) {
    constexpr int kQ = kC / 4;
    const int b0 = 32 * w + (lane & 16), c = lane & 15;
    float y[kQ];  // beta_j t_j of this column
    float4 row[kQ / 4];
    float own, be;
    auto load = [&](int r) {  // row r up to the diagonal, broadcast
        const float* a = A + (b0 + r) * kLd + b0;
#pragma unroll
        for (int j = 0; j < r; j += 4) row[j / 4] = ld_f4(a + j);
        own = a[c];
        be = beta[b0 + r];
    };
    y[0] = 0.f;
    load(1);
#pragma unroll
    for (int r = 1; r < kQ; ++r) {
        float s[4] = {own, 0.f, 0.f, 0.f};
        float last = 0.f;
#pragma unroll
        for (int j = 0; j < r; ++j) {
            const float v = j % 4 == 0 ? row[j / 4].x : j % 4 == 1 ? row[j / 4].y : j % 4 == 2 ? row[j / 4].z : row[j / 4].w;
            if (j < r - 1)
                s[j & 3] = fmaf(v, y[j], s[j & 3]);
            else
                last = v;
        }
        const float b = be;
        if (r + 1 < kQ) load(r + 1);
        const float sum = (s[0] + s[1]) + (s[2] + s[3]);
        const float x = r > c ? -fmaf(last, y[r - 1], sum) : 0.f;
        __syncwarp();  // the row has been read
        A[(b0 + r) * kLd + b0 + c] = x;
        y[r] = b * x;
    }
}

// The joins: the first two warps do the work, all threads of the block call it; the diagonal blocks and the rest of A are
// complete before, t after.
__device__ __forceinline__ void solve_joins(float* A, const float* beta, int tid) {
    constexpr int kH = kC / 2, kQ = kC / 4;
    if (tid < 32) {  // pair p: rows 32 p + 16 + r + 4 j, columns 32 p + c .. c + 3
        const int b = kH * (tid >> 4), r = (tid >> 2) & 3, c = 4 * (tid & 3);
        float* row = A + (b + kQ + r) * kLd + b;
        F4 z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = get4(row + 4 * j * kLd + c);
        acc_tile<0, 4>(z, row, beta + b, A + b * kLd + b + c, 0, kQ);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) put4(row + 4 * j * kLd + c, z[j]);
        __syncwarp();
        acc_tile<0, 4>(z, row + kQ, beta + b + kQ, A + (b + kQ) * kLd + b + c, 0, kQ);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) put4(row + 4 * j * kLd + c, z[j], -1.f);
    }
    __syncthreads();
    // rows 32 + r + 8 j, 16 columns to a warp, four to a thread; t11 and t22 are lower triangular
    const int half = kQ * (tid >> 5), r = (tid >> 2) & 7, c = half + 4 * (tid & 3);
    float* row = A + (kH + r) * kLd;
    F4 z[4];
    if (tid < 64) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = get4(row + 8 * j * kLd + c);
        acc_tile<0, 8>(z, row, beta, A + c, half, kH);
    }
    __syncthreads();
    if (tid < 64) {
#pragma unroll
        for (int j = 0; j < 4; ++j) put4(row + 8 * j * kLd + c, z[j]);
        __syncwarp();  // a warp reads the columns that it wrote
        acc_tile<0, 8>(z, row + kH, beta + kH, A + kH * kLd + c, 0, kQ);
        acc_tile<2, 8>(z, row + kH, beta + kH, A + kH * kLd + c, kQ, kH);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) put4(row + 8 * j * kLd + c, z[j], -1.f);
    }
    __syncthreads();
}

// Byte offsets of the workspace regions of one call (256-byte aligned).
struct Layout {
    size_t rec;     // [BH][M][kRec] fp32 gate records
    // [BH][M][64][64] fp32; tensor cores: bf16 tiles, hi and lo, of t beta and P beta (columns scaled), for the gradient
    // of t beta, P and beta t (rows scaled)
    size_t t, P;
    // The gradient's, fp32 (tensor cores: bf16 tiles of transposed matrices, X and Y as lo and hi parts):
    size_t X, Y;    // [BH][M * 64][Dv]
    size_t S, dS;   // [BH][M][Dk][Dv]: the state entering each chunk, the gradient leaving it
    // Tensor cores, segs > 1 segments of cps chunks to a head (fp32 Dk x Dv records [BH][segs]): the state that a
    // segment adds (B) and the map that it applies to the state entering it (M); the states entering the segments; and
    // for the gradient, what a segment adds to the state's gradient (B2) and the gradients leaving the segments.
    int segs, cps;
    size_t segB, segM, segS, segB2, segdS;
    size_t bytes;
};
Layout layout(const la_shape& s, bool bwd);

struct FwdArgs {
    const void *q, *k, *v, *g, *beta;
    const float* S0;
    void* o;
    float* S;
};
struct BwdArgs {
    const void *q, *k, *v, *g, *beta, *dout;
    void *dq, *dk, *dv, *dg, *dbeta;
    const float *S0, *dS;  // the state before the first position, the gradient of the one after the last; null: zero
    float* dS0;            // null: not wanted
};
// fp32, any head size, on the CUDA cores.
cudaError_t simt_fwd(const FwdArgs& a, const la_shape& s, char* ws, cudaStream_t st);
cudaError_t simt_bwd(const BwdArgs& a, const la_shape& s, char* ws, cudaStream_t st);
// bf16, on the tensor cores: heads are padded on chip to 64 or 128 in both dimensions (tc_dim).
bool tc_ok(const la_shape& s);
int tc_dim(const la_shape& s);
// When the last of n1 blocks of t1 us and then n2 of t2 us ends, one block to each of 152 SMs, taken in order.
double finish(long long n1, double t1, long long n2, double t2);
// Segments of a head for M chunks (a function of the sizes alone).
int tc_segments(const la_shape& s, bool bwd);
cudaError_t tc_fwd(const FwdArgs& a, const la_shape& s, char* ws, cudaStream_t st);
cudaError_t tc_bwd(const BwdArgs& a, const la_shape& s, char* ws, cudaStream_t st);
cudaError_t step(const void* q, const void* k, const void* v, const void* g, const void* beta, float* S, void* out,
                 const la_shape& s, cudaStream_t st);

}  // namespace gd
}  // namespace la
