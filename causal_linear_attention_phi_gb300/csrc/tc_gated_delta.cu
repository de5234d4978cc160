// tc_gated_delta.cu -- tensor-core (tcgen05 / TMEM / TMA) kernels of the gated delta rule for bf16 heads (formulas in
// gated_delta.cuh), chunks of 64 positions.  Heads run at D = 64 or 128 in both dimensions, the smaller that holds
// them: the columns past the true sizes lie outside the tensor maps, arrive as zeros and are not stored.
//
// tc_gd_prepare (one block per chunk): [Q; K] K^T as one 128 x 64 product, the decays applied, t solved for in fp32;
// t and P go to the workspace as bf16 hi + lo tiles in the swizzled layout that the products read.
//
// tc_gd_states (one block per head and segment of chunks): the recurrence with the state transposed, S^T
// [Dv lanes x Dk], so that every product has 128 rows and its left operand comes from TMEM, written there by the
// thread that owns the row:
//   Y^T  = S^T K^T                            R^T = V^T - gam Y^T          (a column is a position)
//   X^T  = R^T + R^T (t beta)^T               (u = beta X)
//   S^T <- gam_C S^T + (tail beta X)^T K      O^T = gam (S^T Q^T) + X^T (P beta)^T
// The fp32 state stays in registers (a quarter of a row to a thread).  Inputs K, Q are bf16 already; what is formed
// here (S, R, X, t, P) enters the products as hi + lo bf16 parts, x = hi + lo to 2^-17, except the S of
// S^T Q^T, which meets one rounding only (it adds 0.5e-3 to the 1.7e-3 of rounding o itself; with
// single parts throughout, correlated keys lift o's error to 7e-3 and the state's to 4e-3).
// Bound by its chain: a chunk's products depend on each other, and each costs its issue, 64 cycles or more a step and a
// round trip through TMEM and registers.  Measured at D = 128: 2.6 us a chunk with outputs, 2.2 us for a segment's sum or
// map (1.9 and 1.45 us at D = 64), against 0.9 us of products; so a sequence is cut into segments, walked at the
// same time (tc_segments).
//
// Roles (576 threads): warp 0 issues TMA, warp 1 tcgen05.mma, warps 2-17 compute: warp w serves TMEM lanes
// 32 (w % 4) .. +31 (value columns r) and, by its group of four, 16 positions and D / 4 state columns of them.
// Every wait is bounded: one that runs out records LA_ERR_TIMEOUT and its thread waits no more, so every role ends.
#include <cudaTypedefs.h>

#include "tc_gated_delta_states.cuh"

namespace la {
namespace gd {
namespace {
using namespace sm100;
using namespace tcgd;

// ------------------------------------------------------------------ t and P of every chunk
// 128 threads, six blocks to an SM: the phases of a chunk are short and each ends in a barrier, so what counts is how many
// chunks an SM has in hand (at B=2 H=16 N=65536 D=128 0.49 ms; with five blocks 0.60, four of 256 threads 0.82).
// Shared memory's data pipe is the busiest unit (58 %): while t is solved for, loads cost the bytes they return.
constexpr int kPrepThreads = 128;
struct PrepSmem {
    // offset 0: blocks of [Q rows 0-63; K rows 64-127] x 64 columns, then (once the product has read them) fp32 A, which
    // becomes t, and P's tiles; t's tiles last, in the place of P's once those are stored (and of A)
    static constexpr int A = 0;
    static constexpr int P = 18432;  // A's bytes rounded up to a tile's alignment
    static constexpr int rec = P + 2 * kBlk;
    static constexpr int bar = rec + kRec * 4;
    static constexpr int total = bar + 32;
};
static_assert(PrepSmem::P >= kC * kLd * 4 && PrepSmem::rec >= 4 * kBlk, "regions");
constexpr size_t kPrepBytes = PrepSmem::total;  // no slack for alignment: it would cost the sixth block
static_assert(6 * (kPrepBytes + 1024) <= 233472, "six blocks to an SM");

// w[x] (columns j0 .. j0 + 31 of row i) times the decay from j to i, 0 outside j <= last (kFull: all inside).  The decays are
// ex2.approx (2^-22 relative) of differences in hi + lo: what they scale enters the products as two bf16 parts (2^-17).
template <bool kResets, bool kFull>
__device__ __forceinline__ void decay32(uint32_t (&w)[32], const float* rec, int i, int j0, int last) {
    const float seg = rec[kSeg + i];
    const float2 hi = make_float2(rec[kGhi + i], rec[kGhi + i]), lo = make_float2(rec[kGlo + i], rec[kGlo + i]);
    const float2 neg = make_float2(-1.f, -1.f);
#pragma unroll
    for (int x = 0; x < 32; x += 4) {
        const F4 gh = get4(rec + kGhi + j0 + x), gl = get4(rec + kGlo + j0 + x);
        const float2 d0 = add2v(fma2v(gh.a, neg, hi), fma2v(gl.a, neg, lo)),
                     d1 = add2v(fma2v(gh.b, neg, hi), fma2v(gl.b, neg, lo));
        const float2 v0 = mul2v(pair(w[x], w[x + 1]), make_float2(ex2_approx(d0.x), ex2_approx(d0.y))),
                     v1 = mul2v(pair(w[x + 2], w[x + 3]), make_float2(ex2_approx(d1.x), ex2_approx(d1.y)));
        const float4 sg = kResets ? ld_f4(rec + kSeg + j0 + x) : make_float4(seg, seg, seg, seg);
        w[x] = (kFull || j0 + x <= last) && sg.x == seg ? __float_as_uint(v0.x) : 0u;
        w[x + 1] = (kFull || j0 + x + 1 <= last) && sg.y == seg ? __float_as_uint(v0.y) : 0u;
        w[x + 2] = (kFull || j0 + x + 2 <= last) && sg.z == seg ? __float_as_uint(v1.x) : 0u;
        w[x + 3] = (kFull || j0 + x + 3 <= last) && sg.w == seg ? __float_as_uint(v1.y) : 0u;
    }
}

template <int D, bool kBwd>
__global__ void __launch_bounds__(kPrepThreads, 6)
tc_gd_prepare(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __nv_bfloat16* __restrict__ g, const __nv_bfloat16* __restrict__ beta, float* __restrict__ recs,
              uint8_t* __restrict__ mats, int N, int M, int* err) {
    extern __shared__ __align__(1024) uint8_t base[];
    if (smem_u32(base) & 1023) {  // the swizzled tiles need it
        if (threadIdx.x == 0) atomicCAS(err, 0, (int)LA_ERR_BOUNDS);
        return;
    }
    float* rec = reinterpret_cast<float*>(base + PrepSmem::rec);
    uint64_t* bar = reinterpret_cast<uint64_t*>(base + PrepSmem::bar);  // loads, product
    uint32_t* slot = reinterpret_cast<uint32_t*>(bar + 2);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, m = blockIdx.x;
    const size_t bh = blockIdx.y, at = bh * M + m;
    const int c0 = m * kC, n = min(kC, N - c0);
    LA_DCHECK(n >= 1 && m < M && (int)gridDim.x == M);
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar + 1, 1);
        fence_mbar_init();
    }
    const uint32_t tmem = enter(slot, 64, warp);
    if (tid == 0) {
        mbar_arrive_expect_tx(bar, 2 * (D / 64) * kBlk);
#pragma unroll
        for (int b = 0; b < D / 64; ++b) {
            tma_load_3d(base + 2 * b * kBlk, &tm_q, 64 * b, c0, (int)bh, bar);
            tma_load_3d(base + (2 * b + 1) * kBlk, &tm_k, 64 * b, c0, (int)bh, bar);
        }
    }
    if (warp == 1) gate_record(g + bh * N, beta + bh * N, c0, n, rec, lane);
    if (tid == 0 && mbar_wait(bar, 0, err, LA_ERR_TIMEOUT)) {
        tc_fence_after();
        constexpr uint32_t id = idesc_bf16_f32(128, kC, 0, 0);
        const uint32_t a = smem_u32(base);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t t = a + (kk >> 2) * 2 * kBlk + (kk & 3) * 32;
            mma_ss(tmem, smem_desc_sw128(t, 16, 1024), smem_desc_sw128(t + kBlk, 16, 1024), id, kk > 0);
        }
        mma_commit(bar + 1);
    }
    const bool ok = mbar_wait(bar + 1, 0, err, LA_ERR_TIMEOUT);
    __syncthreads();  // the gates
    tc_fence_after();
    float* A = reinterpret_cast<float*>(base + PrepSmem::A);
    {
        // lanes 0-63 hold Q K^T, 64-127 K K^T; this thread's row i, 32 columns at a time
        const int i = tid & 63;
        const bool isP = tid < 64, resets = rec[kSeg + kC - 1] != 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
            if (h > (warp & 1)) {  // above the diagonal
#pragma unroll
                for (int x = 0; x < 32; ++x) w[x] = 0u;
            } else {
                tmem_ld32(tmem + ((uint32_t)(32 * warp) << 16) + 32 * h, w);
                tmem_ld_wait();
                const int last = isP ? i : i - 1;
                if (resets)
                    decay32<true, false>(w, rec, i, 32 * h, last);
                else if (h < (warp & 1))
                    decay32<false, true>(w, rec, i, 32 * h, last);
                else
                    decay32<false, false>(w, rec, i, 32 * h, last);
                if (!kBwd && isP) {
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
                        const float4 be = ld_f4(rec + kBeta + 32 * h + x);
                        w[x] = __float_as_uint(be.x * __uint_as_float(w[x]));
                        w[x + 1] = __float_as_uint(be.y * __uint_as_float(w[x + 1]));
                        w[x + 2] = __float_as_uint(be.z * __uint_as_float(w[x + 2]));
                        w[x + 3] = __float_as_uint(be.w * __uint_as_float(w[x + 3]));
                    }
                }
            }
            if (isP) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint4 a, b;
                    split2(__uint_as_float(w[8 * c]), __uint_as_float(w[8 * c + 1]), a.x, b.x);
                    split2(__uint_as_float(w[8 * c + 2]), __uint_as_float(w[8 * c + 3]), a.y, b.y);
                    split2(__uint_as_float(w[8 * c + 4]), __uint_as_float(w[8 * c + 5]), a.z, b.z);
                    split2(__uint_as_float(w[8 * c + 6]), __uint_as_float(w[8 * c + 7]), a.w, b.w);
                    const int off = row_off(i, 4 * h + c);
                    *reinterpret_cast<uint4*>(base + PrepSmem::P + off) = a;
                    *reinterpret_cast<uint4*>(base + PrepSmem::P + kBlk + off) = b;
                }
            } else {
#pragma unroll
                for (int x = 0; x < 32; x += 4)
                    *reinterpret_cast<uint4*>(A + i * kLd + 32 * h + x) = make_uint4(w[x], w[x + 1], w[x + 2], w[x + 3]);
            }
        }
    }
    // a warp of A's rows has all that its diagonal blocks need: it goes on while the other two warps form P
    if (tid >= 64) {
        __syncwarp();
        solve_diagonal(A, rec + kBeta, warp & 1, lane);
    }
    fence_proxy_async_smem();
    __syncthreads();
    uint8_t* mat = mats + at * (size_t)(kBwd ? kMatsBwd : kMatsFwd);
    if (tid == 0) {
        bulk_store(mat + kMatP, base + PrepSmem::P, 2 * kBlk);
        bulk_store(recs + at * kRec, rec, kRec * 4);
        bulk_commit();
    }
    solve_joins(A, rec + kBeta, tid);
    if (tid == 0) bulk_wait_read_all();  // P's tiles have been stored: t's go in their place
    __syncthreads();
    const int i = tid >> 1, j0 = 32 * (tid & 1);
    float4 tr[8];  // half a row
#pragma unroll
    for (int x = 0; x < 8; ++x) tr[x] = ld_f4(A + i * kLd + j0 + 4 * x);
    auto put = [&](uint8_t* tile, auto scale) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 s = scale(2 * c), u = scale(2 * c + 1);
            uint4 a, b;
            split2(s.x, s.y, a.x, b.x);
            split2(s.z, s.w, a.y, b.y);
            split2(u.x, u.y, a.z, b.z);
            split2(u.z, u.w, a.w, b.w);
            const int off = row_off(i, (j0 >> 3) + c);
            *reinterpret_cast<uint4*>(tile + off) = a;
            *reinterpret_cast<uint4*>(tile + kBlk + off) = b;
        }
    };
    put(base + PrepSmem::P, [&](int x) {
        const float4 be = ld_f4(rec + kBeta + j0 + 4 * x);
        return make_float4(tr[x].x * be.x, tr[x].y * be.y, tr[x].z * be.z, tr[x].w * be.w);
    });
    if (kBwd) {
        __syncthreads();  // A has been read
        const float bi = rec[kBeta + i];
        put(base + PrepSmem::A, [&](int x) { return make_float4(bi * tr[x].x, bi * tr[x].y, bi * tr[x].z, bi * tr[x].w); });
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
        bulk_store(mat + kMatF, base + PrepSmem::P, 2 * kBlk);
        if (kBwd) bulk_store(mat + kMatR, base + PrepSmem::A, 2 * kBlk);
        bulk_commit();
        bulk_wait_read_all();  // shared memory outlives the copies' reads; the grid's end makes them visible
        if (!ok) mbar_wait(bar, 0, err, LA_ERR_TIMEOUT);  // never leave with copies in flight
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
}

// ------------------------------------------------------------------ the recurrence
// One block per (segment, head); kSum with D = 128 has a third grid dimension: 0 the sum, 1 the map.
template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
tc_gd_states(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ StateArgs a, int* err) {
    states_block<D, kMode>(tm_q, tm_k, tm_v, a, blockIdx.x, blockIdx.y, kMode == kSum && blockIdx.z == 1, err);
}

// ------------------------------------------------------------------ joining the segments
// Block (slice, head): kCols value columns of the state, carried through the segments' maps in fp32:
// out[p + 1] = B[p] + M[p] out[p], or in reverse out[p - 1] = B[p] + M[p]^T out[p].  A map (64 KB for D = 128) is copied to
// shared memory while the previous one is applied.  A thread forms 2 rows x 4 columns with packed multiply-adds: per
// four terms 6 vector loads from shared memory to 16 of those.
// 32 columns to a block, or 16 or 8 where so many blocks are resident at once (a block's two maps fill most of an SM's shared
// memory), with the terms of a product split between two or four groups of threads: fewer columns read the map less often.
template <int D, int kCols>
struct JoinCfg {
    static constexpr int group = D / 2 * (kCols / 4), split = 32 / kCols, threads = group * split;
    static constexpr int map = D * D * 4;
    static constexpr int S = 2 * map;              // [D][kCols]
    static constexpr int half = S + D * kCols * 4;  // the other groups' sums
    static constexpr int bars = half + (split - 1) * D * kCols * 4;
    static constexpr size_t bytes = bars + 32;
};

template <int D, bool kReverse, int kCols>
__device__ __forceinline__ void join_block(const float* __restrict__ B, const float* __restrict__ Mx,
                                           const float* __restrict__ first, float* __restrict__ out, int P, int Dk, int Dv,
                                           int* err) {
    using L = JoinCfg<D, kCols>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* S = reinterpret_cast<float*>(smem + L::S);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::bars);
    const int tid = threadIdx.x, part = tid / L::group, id = tid % L::group;
    const int row = 2 * (id / (kCols / 4)), c0 = 4 * (id % (kCols / 4)), col = blockIdx.x * kCols + c0;
    float4* half = reinterpret_cast<float4*>(smem + L::half) + id;
    const size_t bh = blockIdx.y, rec = (size_t)D * D;
    LA_DCHECK(col + 3 < D && row + 1 < D && part < L::split);
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar + 1, 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();  // launched with programmatic dependent launch
    // the i-th map applied: segment i, or from the last one back
    auto seg = [&](int i) { return bh * P + (kReverse ? P - 1 - i : i); };
    bool ok = true;
    int issued = 0;
    auto load = [&](int i) {
        if (tid != 0 || !ok) return;
        issued = i + 1;
        mbar_arrive_expect_tx(bar + (i & 1), D * D * 4);
        bulk_load(smem + (i & 1) * L::map, Mx + seg(i) * rec, D * D * 4, bar + (i & 1));
    };
    float4 s[2], b[2];
    auto load_b = [&](int i) {
#pragma unroll
        for (int y = 0; y < 2; ++y) b[y] = ld_f4(B + seg(i) * rec + (row + y) * D + col);
    };
    load(0);
    if (part == 0) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
            s[y] = first && row + y < Dk && col < Dv  // the caller's state or its gradient: true sizes
                       ? ld_f4(first + (bh * Dk + row + y) * Dv + col)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        load_b(0);
    }
    for (int i = 0; i < P; ++i) {
        F4 acc[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            acc[y].a = acc[y].b = make_float2(0.f, 0.f);
            if (part == 0) {
                *reinterpret_cast<float4*>(out + seg(i) * rec + (row + y) * D + col) = s[y];
                *reinterpret_cast<float4*>(S + (row + y) * kCols + c0) = s[y];
                acc[y] = {make_float2(b[y].x, b[y].y), make_float2(b[y].z, b[y].w)};
            }
        }
        if (i == P - 1) break;
        if (i + 1 < P - 1) {
            load(i + 1);  // its buffer was last read before the previous barrier
            if (part == 0) load_b(i + 1);
        }
        ok = ok && mbar_wait(bar + (i & 1), (i >> 1) & 1, err, LA_ERR_TIMEOUT);
        __syncthreads();
        const float* m = reinterpret_cast<const float*>(smem + (i & 1) * L::map);
        const int k0 = part * (D / L::split);
#pragma unroll 4
        for (int kk = 0; kk < D / L::split; kk += 4) {
            const int k = k0 + kk;
            float mv[2][4];
            if (kReverse) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = *reinterpret_cast<const float2*>(m + map_at<D>(k + e, row));
                    mv[0][e] = v.x;
                    mv[1][e] = v.y;
                }
            } else {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float4 v = ld_f4(m + map_at<D>(row + y, k));
                    mv[y][0] = v.x;
                    mv[y][1] = v.y;
                    mv[y][2] = v.z;
                    mv[y][3] = v.w;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 v = ld_f4(S + (k + e) * kCols + c0);
                fma4(acc[0], mv[0][e], v);
                fma4(acc[1], mv[1][e], v);
            }
        }
        if (L::split > 1) {
            if (part > 0) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    half[(2 * (part - 1) + y) * L::group] = make_float4(acc[y].a.x, acc[y].a.y, acc[y].b.x, acc[y].b.y);
            }
            __syncthreads();  // S and the map have been read, the other sums are there
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            s[y] = make_float4(acc[y].a.x, acc[y].a.y, acc[y].b.x, acc[y].b.y);
            if (part == 0) {
#pragma unroll
                for (int o = 0; o < L::split - 1; ++o) {
                    const float4 h = half[(2 * o + y) * L::group];
                    s[y] = make_float4(s[y].x + h.x, s[y].y + h.y, s[y].z + h.z, s[y].w + h.w);
                }
            }
        }
        if (L::split == 1) __syncthreads();  // S and the map have been read
    }
    if (!ok) mbar_drain(bar, 2, issued, err, LA_ERR_TIMEOUT);
}

// The third grid dimension: 0 forwards, 1 in reverse (the gradient's).
template <int D, int kCols>
__global__ void __launch_bounds__(JoinCfg<D, kCols>::threads)
tc_gd_join(const float* __restrict__ B, const float* __restrict__ Mx, const float* __restrict__ first,
           float* __restrict__ out, const float* __restrict__ B2, const float* __restrict__ first2,
           float* __restrict__ out2, int P, int Dk, int Dv, int* err) {
    if (blockIdx.z == 0)
        join_block<D, false, kCols>(B, Mx, first, out, P, Dk, Dv, err);
    else
        join_block<D, true, kCols>(B2, Mx, first2, out2, P, Dk, Dv, err);
}

}  // namespace

namespace tcgd {

template <int D>
cudaError_t prepare(const CUtensorMap& tq, const CUtensorMap& tk, const void* g, const void* beta, float* recs,
                    uint8_t* mats, const la_shape& s, int M, bool bwd, int* err, cudaStream_t st) {
    auto kern = bwd ? tc_gd_prepare<D, true> : tc_gd_prepare<D, false>;
    GD_TRY(allow_smem(kern, kPrepBytes));
    launch_begin("tc_gd_prepare", st);
    const cudaError_t e =
        launch_pdl(kern, dim3(M, s.B * s.H), dim3(kPrepThreads), kPrepBytes, st, tq, tk,
                   (const __nv_bfloat16*)g, (const __nv_bfloat16*)beta, recs, mats, s.N, M, err);
    const cudaError_t e2 = launch_end("tc_gd_prepare", st);
    return e != cudaSuccess ? e : e2;
}
template cudaError_t prepare<64>(const CUtensorMap&, const CUtensorMap&, const void*, const void*, float*, uint8_t*,
                                 const la_shape&, int, bool, int*, cudaStream_t);
template cudaError_t prepare<128>(const CUtensorMap&, const CUtensorMap&, const void*, const void*, float*, uint8_t*,
                                  const la_shape&, int, bool, int*, cudaStream_t);

template <int D>
cudaError_t join(const float* B, const float* Mx, const float* first, float* out, const float* B2, const float* first2,
                 float* out2, int BH, int P, int Dk, int Dv, int* err, cudaStream_t st) {
    const int ways = out2 ? 2 : 1;
    auto go = [&](auto kern, int cols, int threads, size_t smem) {
        GD_TRY(allow_smem(kern, smem));
        launch_begin("tc_gd_join", st);
        const cudaError_t e = launch_pdl(kern, dim3(D / cols, BH, ways), dim3(threads), smem, st, B, Mx, first, out, B2, first2,
                                         out2, P, Dk, Dv, err);
        const cudaError_t e2 = launch_end("tc_gd_join", st);
        return e != cudaSuccess ? e : e2;
    };
    const long long slices = (long long)BH * (D / 16) * ways;
    if (2 * slices <= 152) return go(tc_gd_join<D, 8>, 8, JoinCfg<D, 8>::threads, JoinCfg<D, 8>::bytes);
    if (slices <= 152) return go(tc_gd_join<D, 16>, 16, JoinCfg<D, 16>::threads, JoinCfg<D, 16>::bytes);
    return go(tc_gd_join<D, 32>, 32, JoinCfg<D, 32>::threads, JoinCfg<D, 32>::bytes);
}
template cudaError_t join<64>(const float*, const float*, const float*, float*, const float*, const float*, float*, int,
                              int, int, int, int*, cudaStream_t);
template cudaError_t join<128>(const float*, const float*, const float*, float*, const float*, const float*, float*, int,
                               int, int, int, int*, cudaStream_t);

}  // namespace tcgd

namespace {

template <int D, int kMode>
cudaError_t states(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const StateArgs& a, dim3 grid,
                   int* err, cudaStream_t st) {
    GD_TRY(allow_smem(tc_gd_states<D, kMode>, FwdSmem<D, kMode>::bytes));
    const char* name = kMode == kOut ? "tc_gd_states" : "tc_gd_segments";
    launch_begin(name, st);
    const cudaError_t e =
        launch_pdl(tc_gd_states<D, kMode>, grid, dim3(kThreads), FwdSmem<D, kMode>::bytes, st, tq, tk, tv, a, err);
    const cudaError_t e2 = launch_end(name, st);
    return e != cudaSuccess ? e : e2;
}

template <int D>
cudaError_t fwd(const FwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    const int BH = s.B * s.H, M = (s.N + kC - 1) / kC;
    CUtensorMap tq, tk, tv;
    if (!make_tmap_bf16_rows(&tq, a.q, BH, s.N, s.Dk, kC) || !make_tmap_bf16_rows(&tk, a.k, BH, s.N, s.Dk, kC) ||
        !make_tmap_bf16_rows(&tv, a.v, BH, s.N, s.Dv, kC))
        return cudaErrorInvalidValue;
    int* err = device_error_word();
    const Layout L = layout(s, false);
    float* recs = (float*)(ws + L.rec);
    uint8_t* mats = (uint8_t*)(ws + L.t);
    GD_TRY(prepare<D>(tq, tk, a.g, a.beta, recs, mats, s, M, false, err, st));
    StateArgs sa{};
    sa.recs = recs;
    sa.mats = mats;
    sa.mat_bytes = kMatsFwd;
    sa.M = M;
    sa.P = L.segs;
    sa.cps = L.cps;
    if (L.segs > 1) {
        float *B = (float*)(ws + L.segB), *Mx = (float*)(ws + L.segM), *S = (float*)(ws + L.segS);
        sa.segB = B;
        sa.segM = Mx;
        GD_TRY((states<D, kSum>(tq, tk, tv, sa, dim3(L.segs - 1, BH, D == 128 ? 2 : 1), err, st)));
        GD_TRY(join<D>(B, Mx, a.S0, S, nullptr, nullptr, nullptr, BH, L.segs, s.Dk, s.Dv, err, st));
        sa.S0 = S;
        sa.dk = sa.dv = D;
    } else {
        sa.S0 = a.S0;
        sa.dk = s.Dk;
        sa.dv = s.Dv;
    }
    sa.S_out = a.S;
    sa.o = (__nv_bfloat16*)a.o;
    sa.N = s.N;
    sa.Dk = s.Dk;
    sa.Dv = s.Dv;
    return states<D, kOut>(tq, tk, tv, sa, dim3(L.segs, BH), err, st);
}

}  // namespace

double finish(long long n1, double t1, long long n2, double t2) {
    constexpr int kSms = 152;
    // SMs in two groups of equal time
    double at[2] = {(double)(n1 / kSms + 1) * t1, (double)(n1 / kSms) * t1};
    const long long count[2] = {n1 % kSms, kSms - n1 % kSms};
    if (const long long rounds = n2 / kSms - 2; rounds > 0) {
        n2 -= rounds * kSms;
        at[0] += rounds * t2;
        at[1] += rounds * t2;
    }
    double end = count[0] ? at[0] : at[1];
    while (n2 > 0) {
        const int g = count[0] && at[0] <= at[1] ? 0 : 1;
        at[g] += t2;
        end = at[g] > end ? at[g] : end;
        n2 -= count[g];
    }
    return end;
}

// More segments fill more of the SMs and shorten the chain of chunks, but with P > 1 every segment but the last
// is walked once more for its sum and once for its map (twice the blocks for D = 128), and the segments are joined one
// after another.  The costs are measured microseconds: of a chunk in each kernel, of a block's start, of a step of the
// join.  Predicted and measured, B=2 H=16 N=32768 D=128 gradient without prepare and tc_gd_grads: P = 1 1.82 and 1.80 ms,
// 2 1.71 and 1.69, 4 1.70 and 1.68, 7 1.59 and 1.52, 19 1.76 and 1.73.
int tc_segments(const la_shape& s, bool bwd) {
    const bool wide = tc_dim(s) == 128;
    const long long BH = (long long)s.B * s.H, M = (s.N + kC - 1) / kC;
    const double out = wide ? 2.6 : 1.9, sum = wide ? 2.2 : 1.45;                           // forward; out also kGrad's
    const double rev = bwd ? (wide ? 3.55 : 2.75) : 0., rsum = bwd ? (wide ? 3.0 : 1.95) : 0.;  // adjoint
    const double start = 4.0, launch = 4.0;
    const long long ways = bwd ? 2 : 1, slices = BH * (wide ? 8 : 4) * ways;
    const double step = 2 * slices <= 152 ? (wide ? 1.8 : 0.8)
                                          : (wide ? 3.4 : 1.1) * (slices > 152 ? 1.7 * (double)((slices / 2 + 151) / 152) : 1.0);
    auto walk = [&](long long P, double cps) {  // of every segment
        return finish(bwd ? BH * P : 0, cps * rev + start, BH * P, cps * out + start);
    };
    int best = 1;
    double best_t = walk(1, (double)M);
    for (int P = 2; P <= M && P <= 64; ++P) {
        const long long cps = (M + P - 1) / P;
        if ((M + cps - 1) / cps != P) continue;
        const long long sums = (wide ? 2 : 1) * (P - 1) + (bwd ? 1 : 0);  // the gradient wants the last segment's map too
        const double t = walk(P, (double)cps) + 2 * launch + (P - 1) * step +
                         finish(bwd ? BH * (P - 1) : 0, cps * rsum + start, BH * sums, cps * sum + start);
        if (t < 0.99 * best_t) {
            best_t = t;
            best = P;
        }
    }
    return best;
}

bool tc_ok(const la_shape& s) { return s.dtype == LA_BF16; }
int tc_dim(const la_shape& s) { return s.Dk > 64 || s.Dv > 64 ? 128 : 64; }

cudaError_t tc_fwd(const FwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    return tc_dim(s) == 128 ? fwd<128>(a, s, ws, st) : fwd<64>(a, s, ws, st);
}

}  // namespace gd
}  // namespace la
