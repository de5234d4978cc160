// tc_gated_delta.cu -- tensor-core (tcgen05 / TMEM / TMA) kernels of the gated delta rule for bf16 heads with
// Dk = Dv = 128 or 64 (formulas in gated_delta.cuh), chunks of 64 positions.
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
// The fp32 state stays in registers (half a row to a thread).  Inputs K, Q are bf16 already; what is formed
// here (S, R, X, t, P) enters the products as hi + lo bf16 parts, x = hi + lo to 2^-17, except the S of
// S^T Q^T, which meets one rounding only (it adds 0.5e-3 to the 1.7e-3 of rounding o itself; with
// single parts throughout, correlated keys lift o's error to 7e-3 and the state's to 4e-3).
//
// Roles (576 threads): warp 0 issues TMA, warp 1 tcgen05.mma, warps 2-17 compute: warp w serves TMEM lanes
// 32 (w % 4) .. +31 (value columns r) and, by its group of four, 16 positions and D / 4 state columns of them.
// Every wait is bounded: one that runs out records LA_ERR_TIMEOUT and its thread waits no more, so every role ends.
#include <cudaTypedefs.h>

#include "tc_gated_delta.cuh"

namespace la {
namespace gd {
namespace {
using namespace sm100;
using namespace tcgd;

// ------------------------------------------------------------------ t and P of every chunk
// 128 threads, six blocks to an SM: the phases of a chunk are short and each ends in a barrier, so what counts is how many
// chunks an SM has in hand (256 threads and four blocks: 0.82 ms at B=2 H=16 N=65536 D=128).
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
constexpr size_t kPrepBytes = PrepSmem::total + 1024;

// w[x] (columns j0 .. j0 + 31 of row i) times the decay from j to i, 0 outside j <= last (kFull: all inside).
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
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
struct __align__(8) Bars {
    uint64_t full[2], empty[2];
    uint64_t s_hi, s_lo, y_done, r_hi, r_lo, x_done, u_hi, u_lo, s_done, o_ready, o_done, o_free, final_mma;
};

template <int D, int kMode>
struct FwdSmem {
    static constexpr int tile = D / 64 * kBlk, nmats = kMode == kOut ? kMatsFwd : 2 * kBlk;
    // a stage: K, V, t (and P), Q, gates
    static constexpr int K = 0, V = tile, mats = 2 * tile, Q = mats + nmats, gates = Q + (kMode == kOut ? tile : 0);
    static constexpr int stage = gates + 2048;
    static_assert(kFwdGates <= 2048, "gates");
    static constexpr int out = 2 * stage;  // kGrad: the state's tile and X lo, X hi
    static constexpr int sbytes = D * D * 2, xbytes = 2 * D * 128;
    static constexpr int bars = out + (kMode == kGrad ? sbytes + xbytes : 0);
    static constexpr int slot = bars + 256;
    static constexpr int total = slot + 16;
    static constexpr size_t bytes = total + 1024;
    static_assert(bytes <= 232448, "shared memory");
};

// TMEM columns
template <int D>
struct Tm {
    static constexpr uint32_t SHi = 0, SLo = D / 2, R = D, U = D + 64, O = D + 128;
    // Y, then the two products of X, then dS, each read before the next is written
    static constexpr uint32_t Y = D + 256, X = Y, dS = Y;
    static_assert(dS + 128 <= 512, "TMEM");
};

// Element (row, c) of a segment's map: vectors of four along a row, permuted by the row so that the join's reads of
// eight rows at once meet no bank twice.
template <int D>
__device__ __forceinline__ int map_at(int row, int c) {
    return row * D + ((((c >> 2) ^ ((row >> 1) & 7)) << 2) | (c & 3));
}

// One block per (segment, head); kSum with D = 128 has a third grid dimension: 0 the sum, 1 the map (with D = 64 the
// upper lanes, which have no value columns, carry the map).
template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
tc_gd_states(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, StateArgs a, int* err) {
    using L = FwdSmem<D, kMode>;
    using T = Tm<D>;
    constexpr int kSc = D / kHs;  // state columns of a thread
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars* bar = reinterpret_cast<Bars*>(base + L::bars);
    uint32_t* slot = reinterpret_cast<uint32_t*>(base + L::slot);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int p = blockIdx.x, bh = blockIdx.y, M = a.M, cbeg = p * a.cps, nloc = min(M, cbeg + a.cps) - cbeg;
    const bool map = kMode == kSum && blockIdx.z == 1;  // D = 128: this block forms the segment's map
    LA_DCHECK(nloc >= 1);
    if (kMode == kSum && D == 128 && !map && p >= a.nsum) return;

    if (tid == 0) {
        mbar_init(&bar->full[0], 1);
        mbar_init(&bar->full[1], 1);
        mbar_init(&bar->empty[0], 1 + kWarps);
        mbar_init(&bar->empty[1], 1 + kWarps);
        mbar_init(&bar->s_hi, kWarps);
        mbar_init(&bar->s_lo, kWarps);
        mbar_init(&bar->y_done, 1);
        mbar_init(&bar->r_hi, kWarps);
        mbar_init(&bar->r_lo, kWarps);
        mbar_init(&bar->x_done, 1);
        mbar_init(&bar->u_hi, kWarps);
        mbar_init(&bar->u_lo, kWarps);
        mbar_init(&bar->s_done, 1);
        mbar_init(&bar->o_ready, kWarps);
        mbar_init(&bar->o_done, 1);
        mbar_init(&bar->o_free, kWarps);
        mbar_init(&bar->final_mma, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_q);
    }
    const uint32_t tmem = enter(slot, 512, warp);

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int armed[2] = {-1, -1};
            for (int i = 0; i < nloc; ++i) {
                const int s = i & 1, c = cbeg + i, t0 = c * kC;
                uint8_t* st = base + s * L::stage;
                if (!mbar_wait(&bar->empty[s], ((i >> 1) & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                mbar_arrive_expect_tx(&bar->full[s], (kMode == kOut ? 3 : 2) * L::tile + L::nmats + kFwdGates);
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
                    tma_load_3d(st + L::K + b * kBlk, &tm_k, 64 * b, t0, bh, &bar->full[s]);
                    tma_load_3d(st + L::V + b * kBlk, &tm_v, 64 * b, t0, bh, &bar->full[s]);
                    if (kMode == kOut) tma_load_3d(st + L::Q + b * kBlk, &tm_q, 64 * b, t0, bh, &bar->full[s]);
                }
                const size_t at = (size_t)bh * M + c;
                bulk_load(st + L::mats, a.mats + at * a.mat_bytes, L::nmats, &bar->full[s]);
                bulk_load(st + L::gates, a.recs + at * kRec, kFwdGates, &bar->full[s]);
                armed[s] = i;
            }
            // never leave with copies in flight: wait for the last armed phase of each stage
            for (int s = 0; s < 2; ++s)
                if (armed[s] >= 0) mbar_wait(&bar->full[s], (armed[s] >> 1) & 1, err, LA_ERR_TIMEOUT);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        {
            const uint32_t lead = elect_one();
            constexpr uint32_t id_k = idesc_bf16_f32(128, kC, 0, 0);   // [128 x 64], B K-major
            constexpr uint32_t id_k2 = idesc_bf16_f32(128, 2 * kC, 0, 0);  // [128 x 128]
            constexpr uint32_t id_mn = idesc_bf16_f32(128, D, 0, 1);  // [128 x D], B MN-major
            bool ok = true;
            auto wait = [&](uint64_t* b, int parity) {
                ok = ok && mbar_wait(b, parity, err, LA_ERR_TIMEOUT);
                __syncwarp();
                tc_fence_after();
            };
            // X (P beta)^T of chunk j, added to O (scaled by gam) in two columns' sets, while the next chunk's R is formed
            auto outputs = [&](int j) {
                const uint32_t dP = tile_desc(smem_u32(base + (j & 1) * L::stage) + L::mats + kMatP);
                wait(&bar->o_ready, j & 1);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // X_hi [P_hi; P_lo]^T
                    mma_ts1(lead, tmem + T::O, tmem + T::U + 8 * kk, dP + step_k(kk), id_k2, 1);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts1(lead, tmem + T::O, tmem + T::U + 32 + 8 * kk, dP + step_k(kk), id_k, 1);
                commit1(lead, &bar->o_done);
                commit1(lead, &bar->empty[j & 1]);
            };
            for (int i = 0; i < nloc; ++i) {
                const int s = i & 1, ph = i & 1;
                const uint32_t sg = smem_u32(base + s * L::stage);
                const uint32_t dK = tile_desc(sg + L::K), dQ = tile_desc(sg + L::Q), dM = tile_desc(sg + L::mats);
                const uint32_t dKmn = tile_desc<kBlk>(sg + L::K);
                wait(&bar->full[s], (i >> 1) & 1);
                wait(&bar->s_hi, ph);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)  // Y = S K^T
                    mma_ts1(lead, tmem + T::Y, tmem + T::SHi + 8 * kk, dK + step_k(kk), id_k, kk > 0);
                wait(&bar->s_lo, ph);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ts1(lead, tmem + T::Y, tmem + T::SLo + 8 * kk, dK + step_k(kk), id_k, 1);
                commit1(lead, &bar->y_done);
                if (kMode == kOut && i > 0) outputs(i - 1);
                wait(&bar->r_hi, ph);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // R_hi [t_hi; t_lo]^T: two products of 64 columns
                    mma_ts1(lead, tmem + T::X, tmem + T::R + 8 * kk, dM + step_k(kk), id_k2, kk > 0);
                wait(&bar->r_lo, ph);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts1(lead, tmem + T::X, tmem + T::R + 32 + 8 * kk, dM + step_k(kk), id_k, 1);
                commit1(lead, &bar->x_done);
                if constexpr (kMode == kOut) {  // O = S Q^T, while X is formed
                    if (i > 0) wait(&bar->o_free, ph ^ 1);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ts1(lead, tmem + T::O, tmem + T::SHi + 8 * kk, dQ + step_k(kk), id_k, kk > 0);
                }
                wait(&bar->u_hi, ph);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // the chunk's writes (tail beta X) K
                    mma_ts1(lead, tmem + T::dS, tmem + T::R + 8 * kk, dKmn + step_mn(kk), id_mn, kk > 0);
                wait(&bar->u_lo, ph);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts1(lead, tmem + T::dS, tmem + T::R + 32 + 8 * kk, dKmn + step_mn(kk), id_mn, 1);
                commit1(lead, &bar->s_done);
                if (kMode != kOut) commit1(lead, &bar->empty[s]);
            }
            if (kMode == kOut) outputs(nloc - 1);
            // drain: every MMA this thread issued has completed before TMEM is released
            commit1(lead, &bar->final_mma);
            mbar_wait(&bar->final_mma, 0, err, LA_ERR_TIMEOUT);
        }
    } else {
        // ------------------------------------------------------------ compute warps
        const int ct = tid - 64, h = ct >> 7;        // group: positions kTok h .., state columns kSc h ..
        const int r = 32 * (warp & 3) + lane;        // TMEM lane: value column
        const uint32_t lb = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        bool ok = true;
        auto wait = [&](uint64_t* b, int parity) {
            ok = ok && mbar_wait(b, parity, err, LA_ERR_TIMEOUT);
            __syncwarp();
            tc_fence_after();
        };
        auto arrive = [&](uint64_t* b) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        float2 S[kSc / 2];
#pragma unroll
        for (int x = 0; x < kSc / 2; ++x) {
            const int c = kSc * h + 2 * x;
            if (kMode == kSum) {
                const int d = map ? r : D == 64 ? r - D : -1;
                S[x] = make_float2(c == d ? 1.f : 0.f, c + 1 == d ? 1.f : 0.f);
            } else {
                // the caller's state has the true sizes, the segments' the padded ones
                const float* s0 = a.S0 + (((size_t)bh * a.P + p) * a.dk + c) * a.dv + r;
                S[x] = a.S0 && r < a.dv && c < a.dk ? make_float2(s0[0], s0[a.dv]) : make_float2(0.f, 0.f);
            }
        }
        {
            uint32_t hi[kSc / 2];
            put_hi(lb + T::SHi + kSc / 2 * h, S, hi);
            arrive(&bar->s_hi);
            put_lo(lb + T::SLo + kSc / 2 * h, S, hi);
            arrive(&bar->s_lo);
        }
        // o of chunk j: a warp's store of a position is 64 contiguous bytes (staged for a TMA store it took two
        // barriers of all compute warps in the chain of chunks)
        auto output = [&](int j) {
            wait(&bar->o_done, j & 1);
            uint32_t w[kTok], w2[kTok];
            ld(lb + T::O + kTok * h, w);
            ld(lb + T::O + kC + kTok * h, w2);
            tmem_ld_wait();
            arrive(&bar->o_free);
            const int t0 = (cbeg + j) * kC + kTok * h, n = a.N - t0;
            __nv_bfloat16* o = a.o + ((size_t)bh * a.N + t0) * a.Dv + r;
            if (r < a.Dv) {
#pragma unroll
                for (int x = 0; x < kTok; ++x)
                    if (x < n) o[x * a.Dv] = __float2bfloat16_rn(__uint_as_float(w[x]) + __uint_as_float(w2[x]));
            }
        };
        for (int i = 0; i < nloc; ++i) {
            const int s = i & 1, ph = i & 1;
            uint8_t* sg = base + s * L::stage;
            const float* gates = reinterpret_cast<const float*>(sg + L::gates);
            // a gate of this thread's positions x .. x + 3
            auto gate = [&](int which, int x) { return get4(gates + which + kTok * h + x); };
            float2 R[kTok / 2];  // V, then R, then X; positions in pairs
            uint32_t w[kTok], hi[kTok / 2];
            wait(&bar->full[s], (i >> 1) & 1);
            if (map || 32 * (warp & 3) >= D) {
#pragma unroll
                for (int x = 0; x < kTok / 2; ++x) R[x] = make_float2(0.f, 0.f);
            } else {
                const uint32_t vc = col_addr(sg + L::V, r, kTok * h);
#pragma unroll
                for (int x = 0; x < kTok; x += 2) R[x / 2] = make_float2(col_get(vc, x), col_get(vc, x + 1));
            }
            wait(&bar->y_done, ph);
            ld(lb + T::Y + kTok * h, w);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < kTok; x += 4) {
                const F4 g = gate(kNg, x);
                R[x / 2] = fma2v(g.a, pair(w[x], w[x + 1]), R[x / 2]);
                R[x / 2 + 1] = fma2v(g.b, pair(w[x + 2], w[x + 3]), R[x / 2 + 1]);
            }
            put_hi(lb + T::R + kTok / 2 * h, R, hi);
            arrive(&bar->r_hi);
            put_lo(lb + T::R + 32 + kTok / 2 * h, R, hi);
            arrive(&bar->r_lo);
            if (kMode == kOut && i > 0) output(i - 1);
            wait(&bar->x_done, ph);
            {
                float2 u[kTok / 2];  // tail beta X
                {
                    uint32_t w2[kTok];
                    ld(lb + T::X + kTok * h, w);
                    ld(lb + T::X + kC + kTok * h, w2);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < kTok; x += 2)
                        R[x / 2] = add2v(R[x / 2], add2v(pair(w[x], w[x + 1]), pair(w2[x], w2[x + 1])));
                }
#pragma unroll
                for (int x = 0; x < kTok; x += 4) {
                    const F4 t = gate(kTb, x);
                    u[x / 2] = mul2v(t.a, R[x / 2]);
                    u[x / 2 + 1] = mul2v(t.b, R[x / 2 + 1]);
                }
                put_hi(lb + T::R + kTok / 2 * h, u, hi);
                arrive(&bar->u_hi);
                put_lo(lb + T::R + 32 + kTok / 2 * h, u, hi);
                arrive(&bar->u_lo);
            }
            if constexpr (kMode == kOut) {
                // X for the outputs (its columns are free: the previous chunk's output was read)
                uint32_t lo[kTok / 2];
#pragma unroll
                for (int x = 0; x < kTok / 2; ++x) {
                    hi[x] = hi2(R[x]);
                    lo[x] = lo2(R[x], hi[x]);
                }
                st(lb + T::U + kTok / 2 * h, hi);
                st(lb + T::U + 32 + kTok / 2 * h, lo);
            } else if constexpr (kMode == kGrad) {  // this thread's row of the state's tile (the state entering the chunk) and of X's tiles
                if (ct == 0) bulk_wait_read_all();  // the previous chunk's stores have read the tiles
                named_barrier(1, 32 * kWarps);
                if (r < D) {
                    uint8_t *sS = base + L::out, *sX = sS + L::sbytes;
#pragma unroll
                    for (int x = 0; x < kSc / 2; x += 4) {
                        const int c = kSc * h + 2 * x;
                        *reinterpret_cast<uint4*>(sS + (c >> 6) * (D * 128) + row_off(r, c >> 3)) =
                            make_uint4(hi2(S[x]), hi2(S[x + 1]), hi2(S[x + 2]), hi2(S[x + 3]));
                    }
#pragma unroll
                    for (int x = 0; x < kTok / 2; x += 4) {
                        const uint4 a = make_uint4(hi2(R[x]), hi2(R[x + 1]), hi2(R[x + 2]), hi2(R[x + 3]));
                        const int off = row_off(r, (kTok * h + 2 * x) >> 3);
                        *reinterpret_cast<uint4*>(sX + off) =
                            make_uint4(lo2(R[x], a.x), lo2(R[x + 1], a.y), lo2(R[x + 2], a.z), lo2(R[x + 3], a.w));
                        *reinterpret_cast<uint4*>(sX + D * 128 + off) = a;
                    }
                }
                fence_proxy_async_smem();
                named_barrier(1, 32 * kWarps);
                if (ct == 0) {
                    const size_t at = (size_t)bh * M + cbeg + i;
                    bulk_store(a.s_tiles + at * L::sbytes, base + L::out, L::sbytes);
                    bulk_store(a.x_tiles + at * L::xbytes, base + L::out + L::sbytes, L::xbytes);
                    bulk_commit();
                }
            }
            const float gc = gates[kGam + kC - 1];
            wait(&bar->s_done, ph);
            {
                // half of the columns are updated while the other half are read
                constexpr int kH = kSc / 2;
                uint32_t d0[kH], d1[kH], sh[kH];
                const float2 g2 = make_float2(gc, gc);
                ld(lb + T::dS + kSc * h, d0);
                tmem_ld_wait();
                ld(lb + T::dS + kSc * h + kH, d1);
#pragma unroll
                for (int x = 0; x < kH / 2; ++x) {
                    S[x] = fma2v(g2, S[x], pair(d0[2 * x], d0[2 * x + 1]));
                    sh[x] = hi2(S[x]);
                }
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < kH / 2; ++x) {
                    S[kH / 2 + x] = fma2v(g2, S[kH / 2 + x], pair(d1[2 * x], d1[2 * x + 1]));
                    sh[kH / 2 + x] = hi2(S[kH / 2 + x]);
                }
                st(lb + T::SHi + kH * h, sh);
                tmem_st_wait();
                arrive(&bar->s_hi);
                put_lo(lb + T::SLo + kH * h, S, sh);
                arrive(&bar->s_lo);
            }
            if constexpr (kMode == kOut) {  // S Q^T (complete: issued before dS) scaled in place, the second columns cleared
                ld(lb + T::O + kTok * h, w);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < kTok; x += 4) {
                    const F4 g = gate(kGam, x);
                    const float2 v0 = mul2v(g.a, pair(w[x], w[x + 1])), v1 = mul2v(g.b, pair(w[x + 2], w[x + 3]));
                    w[x] = __float_as_uint(v0.x);
                    w[x + 1] = __float_as_uint(v0.y);
                    w[x + 2] = __float_as_uint(v1.x);
                    w[x + 3] = __float_as_uint(v1.y);
                }
                st(lb + T::O + kTok * h, w);
#pragma unroll
                for (int x = 0; x < kTok; ++x) w[x] = 0u;
                st(lb + T::O + kC + kTok * h, w);
                tmem_st_wait();
                arrive(&bar->o_ready);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->empty[s]);  // this warp is done with V and the gates
        }
        if (kMode == kOut) output(nloc - 1);
        if (ct == 0) bulk_wait_all();
        if (kMode == kSum) {
            const size_t at = ((size_t)bh * a.P + p) * (D * D);
            const int c = r & (D - 1);
#pragma unroll
            for (int x = 0; x < kSc; ++x) {
                const int d = kSc * h + x;
                if (map || r >= D)
                    a.segM[at + map_at<D>(d, c)] = x & 1 ? S[x / 2].y : S[x / 2].x;
                else
                    a.segB[at + d * D + c] = x & 1 ? S[x / 2].y : S[x / 2].x;
            }
        } else if (kMode == kOut && a.S_out && p == a.P - 1 && r < a.Dv) {
#pragma unroll
            for (int x = 0; x < kSc; ++x) {
                const int c = kSc * h + x;
                if (c < a.Dk) a.S_out[((size_t)bh * a.Dk + c) * a.Dv + r] = x & 1 ? S[x / 2].y : S[x / 2].x;
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ joining the segments
// Block (slice, head): kCols value columns of the state, carried through the segments' maps in fp32:
// out[p + 1] = B[p] + M[p] out[p], or in reverse out[p - 1] = B[p] + M[p]^T out[p].  A map (64 KB for D = 128) is copied to
// shared memory while the previous one is applied.  A thread forms 2 rows x 4 columns with packed multiply-adds: per
// four terms 6 vector loads from shared memory to 16 of those.
// 16 columns to a block, with the terms of a product halved between two groups of threads, or 32 columns where that
// many blocks would not be resident at once (a block's two maps fill most of an SM's shared memory).
template <int D, int kCols>
struct JoinCfg {
    static constexpr int group = D / 2 * (kCols / 4), split = 32 / kCols, threads = group * split;
    static constexpr int map = D * D * 4;
    static constexpr int S = 2 * map;              // [D][kCols]
    static constexpr int half = S + D * kCols * 4;  // the second group's sums
    static constexpr int bars = half + (split > 1 ? D * kCols * 4 : 0);
    static constexpr size_t bytes = bars + 32;
};

template <int D, bool kReverse, int kCols>
__global__ void __launch_bounds__(JoinCfg<D, kCols>::threads)
tc_gd_join(const float* __restrict__ B, const float* __restrict__ Mx, const float* __restrict__ first,
           float* __restrict__ out, int P, int Dk, int Dv, int* err) {
    using L = JoinCfg<D, kCols>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* S = reinterpret_cast<float*>(smem + L::S);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::bars);
    const int tid = threadIdx.x, part = tid / L::group, id = tid % L::group;
    const int row = 2 * (id / (kCols / 4)), c0 = 4 * (id % (kCols / 4)), col = blockIdx.x * kCols + c0;
    float4* half = reinterpret_cast<float4*>(smem + L::half) + id;
    const size_t bh = blockIdx.y, rec = (size_t)D * D;
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar + 1, 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();  // launched with programmatic dependent launch
    // the i-th map applied: segment i, or from the last one back
    auto seg = [&](int i) { return bh * P + (kReverse ? P - 1 - i : i); };
    auto load = [&](int i) {
        if (tid != 0) return;
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
            s[y] = !kReverse && first && row + y < Dk && col < Dv  // the caller's state: true sizes
                       ? ld_f4(first + (bh * Dk + row + y) * Dv + col)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        load_b(0);
    }
    bool ok = true;
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
            if (part == 1) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    half[y * L::group] = make_float4(acc[y].a.x, acc[y].a.y, acc[y].b.x, acc[y].b.y);
            }
            __syncthreads();  // S and the map have been read, the second sums are there
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            s[y] = make_float4(acc[y].a.x, acc[y].a.y, acc[y].b.x, acc[y].b.y);
            if (L::split > 1 && part == 0) {
                const float4 h = half[y * L::group];
                s[y] = make_float4(s[y].x + h.x, s[y].y + h.y, s[y].z + h.z, s[y].w + h.w);
            }
        }
        if (L::split == 1) __syncthreads();  // S and the map have been read
    }
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
cudaError_t states(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const StateArgs& a, Mode mode, int BH, int segments, int* err, cudaStream_t st) {
    auto kern = mode == kOut ? tc_gd_states<D, kOut> : mode == kGrad ? tc_gd_states<D, kGrad> : tc_gd_states<D, kSum>;
    const size_t smem = mode == kOut    ? FwdSmem<D, kOut>::bytes
                        : mode == kGrad ? FwdSmem<D, kGrad>::bytes
                                        : FwdSmem<D, kSum>::bytes;
    GD_TRY(allow_smem(kern, smem));
    const char* name = mode == kOut ? "tc_gd_states" : mode == kGrad ? "tc_gd_states_grad" : "tc_gd_segments";
    launch_begin(name, st);
    const cudaError_t e = launch_pdl(kern, dim3(segments, BH, mode == kSum && D == 128 ? 2 : 1), dim3(kThreads), smem, st,
                                     tq, tk, tv, a, err);
    const cudaError_t e2 = launch_end(name, st);
    return e != cudaSuccess ? e : e2;
}

template <int D>
cudaError_t join(const float* B, const float* Mx, const float* first, float* out, int BH, int P, int Dk, int Dv, bool reverse, int* err,
                 cudaStream_t st) {
    const bool wide = (long long)BH * (D / 16) > 152;
    auto kern = reverse ? (wide ? tc_gd_join<D, true, 32> : tc_gd_join<D, true, 16>)
                        : (wide ? tc_gd_join<D, false, 32> : tc_gd_join<D, false, 16>);
    const size_t smem = wide ? JoinCfg<D, 32>::bytes : JoinCfg<D, 16>::bytes;
    GD_TRY(allow_smem(kern, smem));
    const char* name = reverse ? "tc_gd_join_reverse" : "tc_gd_join";
    launch_begin(name, st);
    const cudaError_t e =
        launch_pdl(kern, dim3(D / (wide ? 32 : 16), BH), dim3(wide ? JoinCfg<D, 32>::threads : JoinCfg<D, 16>::threads), smem,
                   st, B, Mx, first, out, P, Dk, Dv, err);
    const cudaError_t e2 = launch_end(name, st);
    return e != cudaSuccess ? e : e2;
}

#define GD_INSTANCE(D)                                                                                              \
    template cudaError_t states<D>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const StateArgs&,    \
                                   Mode, int, int, int*, cudaStream_t);                                            \
    template cudaError_t join<D>(const float*, const float*, const float*, float*, int, int, int, int, bool, int*,     \
                                 cudaStream_t);
GD_INSTANCE(64)
GD_INSTANCE(128)
#undef GD_INSTANCE

}  // namespace tcgd

namespace {

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
        sa.nsum = L.segs - 1;
        GD_TRY(states<D>(tq, tk, tv, sa, kSum, BH, L.segs - 1, err, st));
        GD_TRY(join<D>(B, Mx, a.S0, S, BH, L.segs, s.Dk, s.Dv, false, err, st));
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
    return states<D>(tq, tk, tv, sa, kOut, BH, L.segs, err, st);
}

}  // namespace

// More segments fill more of the 152 SMs and shorten the chain of chunks, but with P > 1 every segment but the last
// is walked once more for its sum and once for its map (twice the blocks for D = 128), and the segments are joined one
// after another.  The costs below are the measured microseconds of a chunk in each kernel.
int tc_segments(const la_shape& s, bool bwd) {
    constexpr int kSms = 152;
    const int BH = s.B * s.H, M = (s.N + kC - 1) / kC;
    const double main = bwd ? 3.8 + 4.6 : 3.2, sum = 2.6, reverse_sum = 2.8, launch = 6.0;
    auto waves = [](long long blocks) { return (double)((blocks + kSms - 1) / kSms); };
    const int D = tc_dim(s);
    const long long slices = (long long)BH * (D / 16);
    const double join = (D == 128 ? 1.9 : 0.8) * (slices > kSms ? 1.6 * waves(slices / 2) : 1.0);
    int best = 1;
    double best_t = waves(BH) * M * main;
    for (int P = 2; P <= M && P <= 64; ++P) {
        const int cps = (M + P - 1) / P;
        if ((M + cps - 1) / cps != P) continue;
        double t = waves((long long)BH * P) * cps * main + 2 * launch + (bwd ? 2 : 1) * P * join;
        t += waves((long long)BH * (P - 1) * (D == 128 ? 2 : 1)) * cps * sum;
        if (bwd) t += waves((long long)BH * (P - 1)) * cps * reverse_sum + 2 * launch;
        if (t < 0.97 * best_t) {
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
