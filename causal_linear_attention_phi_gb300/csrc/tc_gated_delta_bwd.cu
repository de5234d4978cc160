// tc_gated_delta_bwd.cu -- tensor-core gradient of the gated delta rule for bf16 heads, padded on
// chip to D = 128 or 64 (formulas in gated_delta.cuh, layouts in tc_gated_delta.cuh).
//
// tc_gd_sweeps (one block per head, segment and direction): the forward recurrence once more, for the states and X that
// tc_gd_grads needs (tc_gated_delta_states.cuh), and the adjoint recurrence from the last chunk back, transposed like the
// forward one, with dS'^T [Dv lanes x Dk] in registers:
//   dU^T = tail (dS'^T K^T) + dO^T P        Y^T = dU^T + dU^T (beta t)      dV^T = beta Y^T
//   dS^T = gam_C dS'^T + (gam dO)^T Q - (beta gam Y)^T K
// What is formed here enters the products as hi + lo bf16 parts, as in the forward kernel.  It writes dV and,
// for tc_gd_grads, the tiles of Y^T [Dv rows x 64 positions], lo and hi, and of dS'^T [Dv rows x Dk], rounded to bf16
// once like S: a relative error of 2^-9 of each term of the products with the states (S Y^T takes Y's hi part alone, for the
// same size of error).  In dq and dk these terms cancel by little.  dg is what they leave when they cancel: off by 5e-3 of its
// largest for independent keys, more as keys coincide (0.4 with all keys within 0.05 of one direction, beta = 1 and no
// decay; the fp32 path 2e-4).  A second part of S and dS' would add 64 KB to a chunk's tiles, for which shared memory has no room.
//
// tc_gd_grads (persistent blocks, a chunk at a time): with G = Y X^T, F^T = X dO^T, all products with 128 rows,
//   F_ij = (dO_i . X_j) beta_j Gam_ij (i >= j),  E_ij = -beta_i beta_j Gam_ij G_ij (i > j),  dbeta_i = G_ii
//   dQ^T = gam S dO^T + K^T F^T              dK^T = -beta gam S Y^T + tail beta dS' X^T + Q^T F + K^T (E + E^T)^T
// F and E enter as hi + lo parts: dg is a difference of sums over them.  Lanes 0-63 hold E's rows, 64-127 F^T's.
// tc_gd_sweeps is bound by its chain like the forward kernel: 3.55 us a chunk of the adjoint at D = 128 (2.75 at 64).
// tc_gd_grads reads 128 KB of stored tiles and 50 KB of inputs to a chunk of D = 128 and writes 32 KB: B=2 H=16 N=32768
// takes 0.77 ms, 0.66 of the copy rate; the next chunk's tiles are loaded under this one's phases, which are what is left.
#include <cudaTypedefs.h>

#include "tc_gated_delta_states.cuh"

namespace la {
namespace gd {
namespace {
using namespace sm100;
using namespace tcgd;

// ------------------------------------------------------------------ the adjoint recurrence
struct __align__(8) RBars {
    uint64_t full[2], empty[2];
    uint64_t s_hi, s_lo, a_done, g_ready, b_hi, b_lo, y_done, r_hi, r_lo, s_done, final_mma;
};

template <int D>
struct RevSmem {
    static constexpr int tile = D / 64 * kBlk;
    static constexpr int K = 0, Q = tile, dO = 2 * tile, mats = 3 * tile;  // P, then beta t
    static constexpr int gates = mats + 4 * kBlk;
    static constexpr int stage = gates + 2048;
    static constexpr int out = 2 * stage;  // dS' tile; then dV tile and Y's lo and hi tiles
    static constexpr int sbytes = D * D * 2, ybytes = 2 * D * 128;
    static constexpr int bars = out + (sbytes > tile + ybytes ? sbytes : tile + ybytes);
    static constexpr int slot = bars + 256;
    static constexpr int total = slot + 16;
    static constexpr size_t bytes = total + 1024;
    static_assert(bytes <= 232448, "shared memory");
};

struct ReverseArgs {
    const float* recs;
    const uint8_t* mats;
    uint8_t *y_tiles, *ds_tiles;
    const float* segdS;  // [BH][P] records of ek x ev: the gradients of the segments' last states; null: zero
    int ek, ev;
    float* segB2;        // kSums: [BH][P]
    float* dS0;          // [BH] Dk x Dv: the gradient of the first state, or null
    int M, P, cps, Dk, Dv;
};

template <int D>
struct RTm {
    static constexpr uint32_t SHi = 0, SLo = D / 2, A1 = D, A2 = D + 64, B = D + 128, G = D + 192, dS = D + 256;
    static constexpr uint32_t Y = A1;  // two products of 64 columns over A1 and A2, read before
    static_assert(dS + 128 <= 512, "TMEM");
};

// kSums: only the gradient that a segment adds to that of the state before it (segB2), from a zero gradient after it.
template <int D, bool kSums>
__device__ __forceinline__ void reverse_block(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_do,
                                              const CUtensorMap& tm_dv, const ReverseArgs& a, int p, int bh, int* err) {
    const float* __restrict__ recs = a.recs;
    const uint8_t* __restrict__ mats = a.mats;
    uint8_t *__restrict__ y_tiles = a.y_tiles, *__restrict__ ds_tiles = a.ds_tiles;
    const int M = a.M, P = a.P, cps = a.cps, Dv = a.Dv;
    using L = RevSmem<D>;
    using T = RTm<D>;
    constexpr int kSc = D / kHs;  // state columns of a thread
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    RBars* bar = reinterpret_cast<RBars*>(base + L::bars);
    uint32_t* slot = reinterpret_cast<uint32_t*>(base + L::slot);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cbeg = p * cps, cend = min(M, cbeg + cps), nloc = cend - cbeg;
    LA_DCHECK(nloc >= 1);
    if (tid == 0) {
        mbar_init(&bar->full[0], 1);
        mbar_init(&bar->full[1], 1);
        mbar_init(&bar->empty[0], 1 + kWarps);
        mbar_init(&bar->empty[1], 1 + kWarps);
        mbar_init(&bar->s_hi, kWarps);
        mbar_init(&bar->s_lo, kWarps);
        mbar_init(&bar->a_done, 1);
        mbar_init(&bar->g_ready, kWarps);
        mbar_init(&bar->b_hi, kWarps);
        mbar_init(&bar->b_lo, kWarps);
        mbar_init(&bar->y_done, 1);
        mbar_init(&bar->r_hi, kWarps);
        mbar_init(&bar->r_lo, kWarps);
        mbar_init(&bar->s_done, 1);
        mbar_init(&bar->final_mma, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_do);
        tma_prefetch_desc(&tm_dv);
    }
    const uint32_t tmem = enter(slot, 512, warp);

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int armed[2] = {-1, -1};
            for (int i = 0; i < nloc; ++i) {
                const int s = i & 1, c = cend - 1 - i, t0 = c * kC;
                uint8_t* st = base + s * L::stage;
                if (!mbar_wait(&bar->empty[s], ((i >> 1) & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                mbar_arrive_expect_tx(&bar->full[s], 3 * L::tile + 4 * kBlk + kRevGates);
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
                    tma_load_3d(st + L::dO + b * kBlk, &tm_do, 64 * b, t0, bh, &bar->full[s]);
                    tma_load_3d(st + L::K + b * kBlk, &tm_k, 64 * b, t0, bh, &bar->full[s]);
                    tma_load_3d(st + L::Q + b * kBlk, &tm_q, 64 * b, t0, bh, &bar->full[s]);
                }
                const size_t at = (size_t)bh * M + c;
                bulk_load(st + L::mats, mats + at * kMatsBwd + kMatP, 4 * kBlk, &bar->full[s]);
                bulk_load(st + L::gates, recs + at * kRec, kRevGates, &bar->full[s]);
                armed[s] = i;
            }
            // never leave with copies in flight: wait for the last armed phase of each stage
            for (int s = 0; s < 2; ++s)
                if (armed[s] >= 0) mbar_wait(&bar->full[s], (armed[s] >> 1) & 1, err, LA_ERR_TIMEOUT);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t lead = elect_one();
        constexpr uint32_t id_k = idesc_bf16_f32(128, kC, 0, 0);        // [128 x 64], B K-major
        constexpr uint32_t id_amn = idesc_bf16_f32(128, kC, 1, 1);      // A (smem) and B MN-major
        constexpr uint32_t id_mn = idesc_bf16_f32(128, kC, 0, 1);       // [128 x 64], B MN-major
        constexpr uint32_t id_mn2 = idesc_bf16_f32(128, 2 * kC, 0, 1);  // [128 x 128]
        constexpr uint32_t id_mnD = idesc_bf16_f32(128, D, 0, 1);       // [128 x D]
        bool ok = true;
        auto wait = [&](uint64_t* b, int parity) {
            ok = ok && mbar_wait(b, parity, err, LA_ERR_TIMEOUT);
            __syncwarp();
            tc_fence_after();
        };
        for (int i = 0; i < nloc; ++i) {
            const int s = i & 1, ph = i & 1;
            const uint32_t sg = smem_u32(base + s * L::stage);
            const uint32_t dK = tile_desc(sg + L::K), dKmn = tile_desc<kBlk>(sg + L::K), dQmn = tile_desc<kBlk>(sg + L::Q);
            const uint32_t dO = tile_desc<kBlk>(sg + L::dO), dM = tile_desc<kBlk>(sg + L::mats),
                           dT = tile_desc<kBlk>(sg + L::mats + 2 * kBlk);
            wait(&bar->full[s], (i >> 1) & 1);
            if (i > 0) wait(&bar->r_lo, ph ^ 1);  // Y, over A1 and A2, has been read
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // dO^T P
                mma_ss1(lead, tmem + T::A2, dO + step_mn(kk), dM + step_mn(kk), id_amn, kk > 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ss1(lead, tmem + T::A2, dO + step_mn(kk), dM + (kBlk >> 4) + step_mn(kk), id_amn, 1);
            wait(&bar->s_hi, ph);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)  // dS'^T K^T
                mma_ts1(lead, tmem + T::A1, tmem + T::SHi + 8 * kk, dK + step_k(kk), id_k, kk > 0);
            wait(&bar->s_lo, ph);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma_ts1(lead, tmem + T::A1, tmem + T::SLo + 8 * kk, dK + step_k(kk), id_k, 1);
            commit1(lead, &bar->a_done);
            wait(&bar->g_ready, ph);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // (gam dO)^T Q
                mma_ts1(lead, tmem + T::dS, tmem + T::G + 8 * kk, dQmn + step_mn(kk), id_mnD, kk > 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ts1(lead, tmem + T::dS, tmem + T::G + 32 + 8 * kk, dQmn + step_mn(kk), id_mnD, 1);
            wait(&bar->b_hi, ph);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // dU_hi^T [(beta t)_hi | (beta t)_lo]: two products of 64 columns
                mma_ts1(lead, tmem + T::Y, tmem + T::B + 8 * kk, dT + step_mn(kk), id_mn2, kk > 0);
            wait(&bar->b_lo, ph);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ts1(lead, tmem + T::Y, tmem + T::B + 32 + 8 * kk, dT + step_mn(kk), id_mn, 1);
            commit1(lead, &bar->y_done);
            wait(&bar->r_hi, ph);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // -(beta gam Y)^T K
                mma_ts1(lead, tmem + T::dS, tmem + T::B + 8 * kk, dKmn + step_mn(kk), id_mnD, 1);
            wait(&bar->r_lo, ph);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ts1(lead, tmem + T::dS, tmem + T::B + 32 + 8 * kk, dKmn + step_mn(kk), id_mnD, 1);
            commit1(lead, &bar->s_done);
            commit1(lead, &bar->empty[s]);
        }
        // drain: every MMA issued has completed before TMEM is released
        commit1(lead, &bar->final_mma);
        mbar_wait(&bar->final_mma, 0, err, LA_ERR_TIMEOUT);
    } else {
        // ------------------------------------------------------------ compute warps
        const int ct = tid - 64, h = ct >> 7;  // group: positions kTok h .., state columns kSc h ..
        const int r = 32 * (warp & 3) + lane;  // TMEM lane: value column
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
            const float* s0 = a.segdS + (((size_t)bh * P + p) * a.ek + c) * a.ev + r;
            S[x] = !kSums && a.segdS && r < a.ev && c < a.ek ? make_float2(s0[0], s0[a.ev]) : make_float2(0.f, 0.f);
        }
        uint8_t* out = base + L::out;
        for (int i = 0; i < nloc; ++i) {
            const int s = i & 1, ph = i & 1, c = cend - 1 - i;
            const size_t at = (size_t)bh * M + c;
            LA_DCHECK(c >= 0 && c < M && bh < (int)gridDim.y);
            uint8_t* sg = base + s * L::stage;
            const float* gates = reinterpret_cast<const float*>(sg + L::gates);
            auto gate = [&](int which, int x) { return get4(gates + which + kTok * h + x); };
            {  // the state gradient's parts, and the signal that they are there
                uint32_t hi[kSc / 2];
                put_hi(lb + T::SHi + kSc / 2 * h, S, hi);
                arrive(&bar->s_hi);
                put_lo(lb + T::SLo + kSc / 2 * h, S, hi);
                arrive(&bar->s_lo);
                if constexpr (!kSums) {  // its tile: the gradient leaving this chunk
                    if (ct == 0) bulk_wait_read_all();
                    named_barrier(1, 32 * kWarps);
                    if (r < D) {
#pragma unroll
                        for (int x = 0; x < kSc; x += 8) {
                            const int cc = kSc * h + x;
                            *reinterpret_cast<uint4*>(out + (cc >> 6) * (D * 128) + row_off(r, cc >> 3)) =
                                make_uint4(hi[x / 2], hi[x / 2 + 1], hi[x / 2 + 2], hi[x / 2 + 3]);
                        }
                    }
                    fence_proxy_async_smem();
                    named_barrier(1, 32 * kWarps);
                    if (ct == 0) {
                        bulk_store(ds_tiles + at * L::sbytes, out, L::sbytes);
                        bulk_commit();
                    }
                }
            }
            uint32_t w[kTok], w2[kTok], hi[kTok / 2];
            wait(&bar->full[s], (i >> 1) & 1);
            {
                uint32_t lo[kTok / 2];
                if (32 * (warp & 3) >= D) {
#pragma unroll
                    for (int x = 0; x < kTok / 2; ++x) hi[x] = lo[x] = 0u;
                } else {
                    const uint32_t dc = col_addr(sg + L::dO, r, kTok * h);
#pragma unroll
                    for (int x = 0; x < kTok; x += 4) {
                        const F4 g = gate(kGam, x);
                        const float2 v0 = mul2v(g.a, make_float2(col_get(dc, x), col_get(dc, x + 1))),
                                     v1 = mul2v(g.b, make_float2(col_get(dc, x + 2), col_get(dc, x + 3)));
                        hi[x / 2] = hi2(v0);
                        lo[x / 2] = lo2(v0, hi[x / 2]);
                        hi[x / 2 + 1] = hi2(v1);
                        lo[x / 2 + 1] = lo2(v1, hi[x / 2 + 1]);
                    }
                }
                st(lb + T::G + kTok / 2 * h, hi);  // free: the previous chunk's products are complete
                st(lb + T::G + 32 + kTok / 2 * h, lo);
                tmem_st_wait();
                arrive(&bar->g_ready);
            }
            float2 dU[kTok / 2];  // dU, then Y; positions in pairs
            wait(&bar->a_done, ph);
            ld(lb + T::A1 + kTok * h, w);
            ld(lb + T::A2 + kTok * h, w2);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < kTok; x += 4) {
                const F4 t = gate(kTail, x);
                dU[x / 2] = fma2v(t.a, pair(w[x], w[x + 1]), pair(w2[x], w2[x + 1]));
                dU[x / 2 + 1] = fma2v(t.b, pair(w[x + 2], w[x + 3]), pair(w2[x + 2], w2[x + 3]));
            }
            put_hi(lb + T::B + kTok / 2 * h, dU, hi);
            arrive(&bar->b_hi);
            put_lo(lb + T::B + 32 + kTok / 2 * h, dU, hi);
            arrive(&bar->b_lo);
            wait(&bar->y_done, ph);
            ld(lb + T::Y + kTok * h, w);
            ld(lb + T::Y + kC + kTok * h, w2);
            tmem_ld_wait();
            float2 b[kTok / 2];  // -beta gam Y
#pragma unroll
            for (int x = 0; x < kTok; x += 4) {
                const F4 bg = gate(kBg, x);
                dU[x / 2] = add2v(dU[x / 2], add2v(pair(w[x], w[x + 1]), pair(w2[x], w2[x + 1])));
                dU[x / 2 + 1] = add2v(dU[x / 2 + 1], add2v(pair(w[x + 2], w[x + 3]), pair(w2[x + 2], w2[x + 3])));
                b[x / 2] = mul2v(bg.a, dU[x / 2]);
                b[x / 2 + 1] = mul2v(bg.b, dU[x / 2 + 1]);
            }
            put_hi(lb + T::B + kTok / 2 * h, b, hi);
            arrive(&bar->r_hi);
            put_lo(lb + T::B + 32 + kTok / 2 * h, b, hi);
            arrive(&bar->r_lo);
            const float gc = gates[kGam + kC - 1];
            if constexpr (!kSums) {
                // dV's tile [positions][value columns] and Y's [value columns][positions]
                if (ct == 0) bulk_wait_read_all();
                named_barrier(1, 32 * kWarps);
                if (r < D) {
                    const uint32_t oc = col_addr(out, r, kTok * h);
#pragma unroll
                    for (int x = 0; x < kTok; x += 4) {
                        const F4 be = gate(kBeta, x);
                        const float2 v0 = mul2v(be.a, dU[x / 2]), v1 = mul2v(be.b, dU[x / 2 + 1]);
                        col_put2(oc, x, v0.x, v0.y);
                        col_put2(oc, x + 2, v1.x, v1.y);
                    }
#pragma unroll
                    for (int x = 0; x < kTok / 2; x += 4) {
                        const uint4 a = make_uint4(hi2(dU[x]), hi2(dU[x + 1]), hi2(dU[x + 2]), hi2(dU[x + 3]));
                        uint8_t* y = out + L::tile + row_off(r, (kTok * h + 2 * x) >> 3);
                        *reinterpret_cast<uint4*>(y) =
                            make_uint4(lo2(dU[x], a.x), lo2(dU[x + 1], a.y), lo2(dU[x + 2], a.z), lo2(dU[x + 3], a.w));
                        *reinterpret_cast<uint4*>(y + D * 128) = a;
                    }
                }
                fence_proxy_async_smem();
                named_barrier(1, 32 * kWarps);
                if (ct == 0) {
#pragma unroll
                    for (int b = 0; b < D / 64; ++b)
                        if (64 * b < Dv) tma_store_3d(&tm_dv, out + b * kBlk, 64 * b, c * kC, bh);
                    bulk_store(y_tiles + at * L::ybytes, out + L::tile, L::ybytes);
                    bulk_commit();
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->empty[s]);  // this warp is done with dO and the gates
            wait(&bar->s_done, ph);
            {
                uint32_t d[kSc];
                const float2 g2 = make_float2(gc, gc);
                ld(lb + T::dS + kSc * h, d);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < kSc / 2; ++x) S[x] = fma2v(g2, S[x], pair(d[2 * x], d[2 * x + 1]));
            }
        }
        if (ct == 0) bulk_wait_all();
        if (kSums && r < D) {
#pragma unroll
            for (int x = 0; x < kSc; ++x)
                a.segB2[(((size_t)bh * P + p) * D + kSc * h + x) * D + r] = x & 1 ? S[x / 2].y : S[x / 2].x;
        }
        if (!kSums && a.dS0 && p == 0 && r < a.Dv) {
#pragma unroll
            for (int x = 0; x < kSc; ++x) {
                const int c = kSc * h + x;
                if (c < a.Dk) a.dS0[((size_t)bh * a.Dk + c) * a.Dv + r] = x & 1 ? S[x / 2].y : S[x / 2].x;
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

// ------------------------------------------------------------------ both recurrences at once
// They do not depend on each other: one grid of both fills the SMs better than two, and its last wave is shorter.  The
// third grid dimension: 0 the adjoint one (the longer), then the forward one, and with kSums and D = 128 its maps.
template <int D, bool kSums>
struct SweepSmem {
    static constexpr size_t fwd = FwdSmem<D, kSums ? kSum : kGrad>::bytes, rev = RevSmem<D>::bytes;
    static constexpr size_t bytes = fwd > rev ? fwd : rev;
};
template <int D, bool kSums>
__global__ void __launch_bounds__(kThreads, 1)
tc_gd_sweeps(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
             const __grid_constant__ CUtensorMap tm_dv, const __grid_constant__ StateArgs a,
             const __grid_constant__ ReverseArgs ra, int* err) {
    const int p = blockIdx.x, bh = blockIdx.y;
    if (blockIdx.z == 0) {
        if (!kSums || p > 0)  // the first segment's sum is not needed
            reverse_block<D, kSums>(tm_q, tm_k, tm_do, tm_dv, ra, p, bh, err);
        return;
    }
    const bool map = kSums && blockIdx.z == 2;
    if (kSums && D == 128 && !map && p >= a.P - 1) return;  // nor the last one's, but its map
    states_block<D, kSums ? kSum : kGrad>(tm_q, tm_k, tm_v, a, p, bh, map, err);
}

// ------------------------------------------------------------------ dq, dk, dg, dbeta of a chunk
template <int D>
struct GradSmem {
    static constexpr int TS = D * 128;  // a tile of D rows x 64 columns
    static constexpr int S = 0, XLo = S + D * D * 2, XHi = XLo + TS, YLo = XHi + TS, Y = YLo + TS, dS = Y + TS;
    static constexpr int QK = dS + D * D * 2;  // blocks of [Q rows; K rows] x 64 columns
    static constexpr int dO = QK + 2 * (D / 64) * kBlk;
    static constexpr int FHi = dO + (D / 64) * kBlk, FLo = FHi + kBlk, EHi = FLo + kBlk, ELo = EHi + kBlk;
    static constexpr int out = FHi;  // dq and dk tiles, once the products have read F and E
    static_assert(2 * (D / 64) * kBlk <= 4 * kBlk, "output tiles");
    static constexpr int rec = ELo + kBlk;
    static constexpr int part = rec + kRec * 4;  // fp32 partial sums, below
    static constexpr int pRow = 0, pCol = pRow + 4 * 128, pTok = pCol + 4 * kC, pSum = pTok + 4 * kC,
                         dBeta = pSum + 2 * kWarps, pEnd = dBeta + kC;
    static constexpr int bars = part + pEnd * 4;
    static constexpr int slot = bars + 128;
    static constexpr int total = slot + 16;
    static constexpr size_t bytes = total + 1024;
    static_assert(bytes <= 232448, "shared memory");
};
struct __align__(8) GBars {
    uint64_t a_full, b_full;    // X, Y, S, dS', dO; Q, K and the gates
    uint64_t a_free, b_free;
    uint64_t pairs_done, pairs_ready, out_done, acc_free;
    uint64_t final_mma;
};
struct GTm {
    static constexpr uint32_t q1 = 0, k1 = 64, k3 = 128;          // S dO^T; S Y^T; dS' X^T as two halves
    static constexpr uint32_t G = 256, FT = 320, kk = 384, qk = 448;
    static constexpr uint32_t q2 = 256, k2 = 384;                 // over the four above, two halves each
};

// v[x] (x < 16) summed over the 32 lanes; lane l (even ones suffice) gets the total of column (l >> 1) & 15.
__device__ __forceinline__ float reduce16(float (&v)[16], int lane) {
#pragma unroll
    for (int o = 16, n = 8; n >= 1; o >>= 1, n >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int x = 0; x < n; ++x) {
            const float send = up ? v[x] : v[x + n];
            const float keep = up ? v[x + n] : v[x];
            v[x] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tc_gd_grads(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_dq,
            const __grid_constant__ CUtensorMap tm_dk, const float* __restrict__ recs,
            const uint8_t* __restrict__ x_tiles, const uint8_t* __restrict__ y_tiles,
            const uint8_t* __restrict__ s_tiles, const uint8_t* __restrict__ ds_tiles, __nv_bfloat16* __restrict__ dg,
            __nv_bfloat16* __restrict__ dbeta, int N, int M, int total, int Dk, int* err) {
    using L = GradSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    GBars* bar = reinterpret_cast<GBars*>(base + L::bars);
    uint32_t* slot = reinterpret_cast<uint32_t*>(base + L::slot);
    float* rec = reinterpret_cast<float*>(base + L::rec);
    float* part = reinterpret_cast<float*>(base + L::part);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nloc = (total - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // chunks of this block
    LA_DCHECK(nloc >= 1);
    if (tid == 0) {
        mbar_init(&bar->a_full, 1);
        mbar_init(&bar->b_full, 1);
        mbar_init(&bar->a_free, 1 + kWarps);
        mbar_init(&bar->b_free, kWarps);
        mbar_init(&bar->pairs_done, 1);
        mbar_init(&bar->pairs_ready, kWarps);
        mbar_init(&bar->out_done, 1);
        mbar_init(&bar->acc_free, kWarps);
        mbar_init(&bar->final_mma, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_do);
        tma_prefetch_desc(&tm_dq);
        tma_prefetch_desc(&tm_dk);
    }
    const uint32_t tmem = enter(slot, 512, warp);
    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int a_armed = -1, b_armed = -1;
            for (int i = 0; i < nloc; ++i) {
                const size_t at = (size_t)blockIdx.x + (size_t)gridDim.x * i;
                const int bh = (int)(at / M), c0 = (int)(at % M) * kC;
                if (!mbar_wait(&bar->a_free, (i & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                mbar_arrive_expect_tx(&bar->a_full, 2 * D * D * 2 + 4 * L::TS + (D / 64) * kBlk);
                bulk_load(base + L::XLo, x_tiles + at * (2 * L::TS), 2 * L::TS, &bar->a_full);
                bulk_load(base + L::YLo, y_tiles + at * (2 * L::TS), 2 * L::TS, &bar->a_full);
#pragma unroll
                for (int b = 0; b < D / 64; ++b)
                    tma_load_3d(base + L::dO + b * kBlk, &tm_do, 64 * b, c0, bh, &bar->a_full);
                bulk_load(base + L::S, s_tiles + at * (D * D * 2), D * D * 2, &bar->a_full);
                bulk_load(base + L::dS, ds_tiles + at * (D * D * 2), D * D * 2, &bar->a_full);
                a_armed = i;
                if (!mbar_wait(&bar->b_free, (i & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                mbar_arrive_expect_tx(&bar->b_full, 2 * (D / 64) * kBlk + kRec * 4);
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
                    tma_load_3d(base + L::QK + 2 * b * kBlk, &tm_q, 64 * b, c0, bh, &bar->b_full);
                    tma_load_3d(base + L::QK + (2 * b + 1) * kBlk, &tm_k, 64 * b, c0, bh, &bar->b_full);
                }
                bulk_load(rec, recs + at * kRec, kRec * 4, &bar->b_full);
                b_armed = i;
            }
            // never leave with copies in flight
            if (a_armed >= 0) mbar_wait(&bar->a_full, a_armed & 1, err, LA_ERR_TIMEOUT);
            if (b_armed >= 0) mbar_wait(&bar->b_full, b_armed & 1, err, LA_ERR_TIMEOUT);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t lead = elect_one();
        bool ok = true;
        auto wait = [&](uint64_t* b, int parity) {
            ok = ok && mbar_wait(b, parity, err, LA_ERR_TIMEOUT);
            __syncwarp();
            tc_fence_after();
        };
        constexpr uint32_t id_kk = idesc_bf16_f32(128, kC, 0, 0), id_mk = idesc_bf16_f32(128, kC, 1, 0),
                           id_mm = idesc_bf16_f32(128, kC, 1, 1), id_mm2 = idesc_bf16_f32(128, 2 * kC, 1, 1),
                           id_mk2 = idesc_bf16_f32(128, 2 * kC, 1, 0);
        const uint32_t b0 = smem_u32(base);
        constexpr int TS = L::TS, kSteps = D / 16;
        const uint32_t dQ = tile_desc(b0 + L::QK), dK = tile_desc(b0 + L::QK + kBlk), dO = tile_desc(b0 + L::dO);
        // MN-major left operands: blocks of 64 rows (of M) one tile apart
        const uint32_t aBelow = tile_desc<TS>(b0 + L::XLo - TS), aLo = tile_desc<TS>(b0 + L::XLo),
                       aHi = tile_desc<TS>(b0 + L::XHi), aYLo = tile_desc<TS>(b0 + L::YLo), aY = tile_desc<TS>(b0 + L::Y),
                       aS = tile_desc<TS>(b0 + L::S), adS = tile_desc<TS>(b0 + L::dS);
        const uint32_t mQ = tile_desc<2 * kBlk>(b0 + L::QK), mK = tile_desc<2 * kBlk>(b0 + L::QK + kBlk);
        const uint32_t fMn = tile_desc<kBlk>(b0 + L::FHi), eMn = tile_desc<kBlk>(b0 + L::EHi);
        const uint32_t fK = tile_desc(b0 + L::FHi), eK = tile_desc(b0 + L::EHi);
        for (int i = 0; i < nloc; ++i) {
            const int ph = i & 1;
            wait(&bar->a_full, ph);
            if (i > 0) wait(&bar->acc_free, ph ^ 1);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)  // lanes 64-127: X dO^T
                mma_ss1(lead, tmem + GTm::FT, aBelow + step_mn(k), dO + step_k(k), id_mk, k > 0);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
                mma_ss1(lead, tmem + GTm::FT, aLo + step_mn(k), dO + step_k(k), id_mk, 1);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)  // lanes 0-63: Y X^T
                mma_ss1(lead, tmem + GTm::G, aY + step_mn(k), aHi + step_mn(k), id_mm, k > 0);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
                mma_ss1(lead, tmem + GTm::G, aY + step_mn(k), aLo + step_mn(k), id_mm, 1);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
                mma_ss1(lead, tmem + GTm::G, aYLo + step_mn(k), aHi + step_mn(k), id_mm, 1);
            wait(&bar->b_full, ph);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)  // lanes 64-127: K Q^T
                mma_ss1(lead, tmem + GTm::qk, dQ + step_k(k, 2 * kBlk), dQ + step_k(k, 2 * kBlk), id_kk, k > 0);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)  // lanes 0-63: K K^T
                mma_ss1(lead, tmem + GTm::kk, dK + step_k(k, 2 * kBlk), dK + step_k(k, 2 * kBlk), id_kk, k > 0);
            commit1(lead, &bar->pairs_done);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)  // S dO^T
                mma_ss1(lead, tmem + GTm::q1, aS + step_mn(k), dO + step_k(k), id_mk, k > 0);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)  // S Y^T
                mma_ss1(lead, tmem + GTm::k1, aS + step_mn(k), aY + step_mn(k), id_mm, k > 0);
#pragma unroll
            for (int k = 0; k < kSteps; ++k)  // dS' [X_lo | X_hi]^T
                mma_ss1(lead, tmem + GTm::k3, adS + step_mn(k), aLo + step_mn(k), id_mm2, k > 0);
            commit1(lead, &bar->a_free);
            wait(&bar->pairs_ready, ph);  // F and E are in their tiles, their products have been read
#pragma unroll
            for (int k = 0; k < 4; ++k)  // K^T F^T, with [F_hi | F_lo]
                mma_ss1(lead, tmem + GTm::q2, mK + step_mn(k), fMn + step_mn(k), id_mm2, k > 0);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // Q^T F
                mma_ss1(lead, tmem + GTm::k2, mQ + step_mn(k), fK + step_k(k), id_mk2, k > 0);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // K^T E^T
                mma_ss1(lead, tmem + GTm::k2, mK + step_mn(k), eK + step_k(k), id_mk2, 1);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // K^T E
                mma_ss1(lead, tmem + GTm::k2, mK + step_mn(k), eMn + step_mn(k), id_mm2, 1);
            commit1(lead, &bar->out_done);
        }
        // drain: every MMA issued has completed before TMEM is released
        commit1(lead, &bar->final_mma);
        mbar_wait(&bar->final_mma, 0, err, LA_ERR_TIMEOUT);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ compute warps
        const int ct = tid - 64, h = ct >> 7, r = 32 * (warp & 3) + lane, q4 = warp & 3;
        const uint32_t lb = tmem + ((uint32_t)(32 * q4) << 16);
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
        const bool isF = r >= kC;
        const int row = r & (kC - 1), col0 = 16 * h;
        for (int i = 0; i < nloc; ++i) {
            const int ph = i & 1;
            const size_t at = (size_t)blockIdx.x + (size_t)gridDim.x * i;
            const int bh = (int)(at / M), c0 = (int)(at % M) * kC, n = min(kC, N - c0);
            LA_DCHECK(at < (size_t)total && n >= 1);
            wait(&bar->a_full, ph);
            float kept = 0.f;  // <dS', S>
#pragma unroll
            for (int x = 0; x < D * D / 8 / (32 * kWarps); ++x) {
                const int o = 16 * (ct + 32 * kWarps * x);
                const uint4 a = *reinterpret_cast<const uint4*>(base + L::S + o);
                const uint4 b = *reinterpret_cast<const uint4*>(base + L::dS + o);
                kept = fmaf(bf_lo(a.x), bf_lo(b.x), fmaf(bf_hi(a.x), bf_hi(b.x), kept));
                kept = fmaf(bf_lo(a.y), bf_lo(b.y), fmaf(bf_hi(a.y), bf_hi(b.y), kept));
                kept = fmaf(bf_lo(a.z), bf_lo(b.z), fmaf(bf_hi(a.z), bf_hi(b.z), kept));
                kept = fmaf(bf_lo(a.w), bf_lo(b.w), fmaf(bf_hi(a.w), bf_hi(b.w), kept));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->a_free);
            // the F and E tiles are free once the previous chunk's stores have read dq and dk out of them, the
            // partial sums once its dg is formed
            if (ct == 0) bulk_wait_read_all();
            named_barrier(1, 32 * kWarps);
            wait(&bar->b_full, ph);
            wait(&bar->pairs_done, ph);
            // F^T (row j, columns i >= j) or E (row i, columns j < i): this thread's 16 columns; none in a block
            // on the other side of the diagonal
            float pr[16], rsum = 0.f;
            uint4 phi[2], plo[2];
            uint32_t* eh = reinterpret_cast<uint32_t*>(phi);
            uint32_t* el = reinterpret_cast<uint32_t*>(plo);
            const int row0 = 32 * (q4 & 1);  // the warp's rows are row0 .. +31
            if (isF ? col0 + 15 >= row0 : col0 <= row0 + 31) {
                uint32_t v[16], pq[16];
                ld(lb + (isF ? GTm::FT : GTm::G) + col0, v);
                ld(lb + (isF ? GTm::qk : GTm::kk) + col0, pq);
                tmem_ld_wait();
                const float seg = rec[kSeg + row], hi = rec[kGhi + row], lo = rec[kGlo + row], br = rec[kBeta + row];
                const float sgn = isF ? -1.f : 1.f;
                const bool resets = rec[kSeg + kC - 1] != 0.f;
#pragma unroll
                for (int x0 = 0; x0 < 16; x0 += 4) {
                    const float4 gh = ld_f4(rec + kGhi + col0 + x0), gl = ld_f4(rec + kGlo + col0 + x0);
                    float4 sg = make_float4(seg, seg, seg, seg), be = make_float4(-1.f, -1.f, -1.f, -1.f);
                    if (resets) sg = ld_f4(rec + kSeg + col0 + x0);
                    if (!isF) be = ld_f4(rec + kBeta + col0 + x0);
                    const float ghv[4] = {gh.x, gh.y, gh.z, gh.w}, glv[4] = {gl.x, gl.y, gl.z, gl.w},
                                sgv[4] = {sg.x, sg.y, sg.z, sg.w}, bev[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int x = x0 + e, col = col0 + x;
                        const float raw = __uint_as_float(v[x]);
                        if (!isF && col == row) part[L::dBeta + row] = raw;
                        const float d = (hi - ghv[e]) + (lo - glv[e]);  // G_row - G_col
                        const bool in = (isF ? col >= row : col < row) && sgv[e] == seg;
                        const float val = in ? raw * (-br * bev[e] * ex2_approx(d * sgn)) : 0.f;
                        v[x] = __float_as_uint(val);
                        pr[x] = in && col != row ? val * __uint_as_float(pq[x]) : 0.f;
                        rsum += pr[x];
                    }
                }
#pragma unroll
                for (int x = 0; x < 16; x += 2)
                    split2(__uint_as_float(v[x]), __uint_as_float(v[x + 1]), eh[x / 2], el[x / 2]);
            } else {
#pragma unroll
                for (int x = 0; x < 16; ++x) pr[x] = 0.f;
                phi[0] = phi[1] = plo[0] = plo[1] = make_uint4(0u, 0u, 0u, 0u);
            }
            uint8_t* tile = base + (isF ? L::FHi : L::EHi);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int off = row_off(row, (col0 >> 3) + x);
                *reinterpret_cast<uint4*>(tile + off) = phi[x];
                *reinterpret_cast<uint4*>(tile + kBlk + off) = plo[x];
            }
            fence_proxy_async_smem();
            arrive(&bar->pairs_ready);
            // shares of dG: a row of E adds to its position, its columns are taken off theirs; F^T the other way round
            part[L::pRow + h * 128 + r] = isF ? -rsum : rsum;
            const float cs = reduce16(pr, lane);
            if ((lane & 1) == 0) part[L::pCol + q4 * kC + col0 + (lane >> 1)] = isF ? cs : -cs;
            wait(&bar->out_done, ph);
            // row r = dk, positions 16 h ..
            float tok[16], outs = 0.f, dq_even = 0.f, dk_even = 0.f;
            const uint32_t sq = col_addr(base + L::out, r & (D - 1), col0), sk = sq + (D / 64) * kBlk;
            const uint32_t qc = col_addr(base + L::QK, r & (D - 1), col0, 2 * kBlk), kc = qc + kBlk;  // [Q; K] blocks
#pragma unroll
            for (int x0 = 0; x0 < 16; x0 += 8) {
                const int t0 = col0 + x0;
                uint32_t q1[8], k1[8], ka[8], kb[8], qa[8], qb[8], ea[8], eb[8];
                ld(lb + GTm::q1 + t0, q1);
                ld(lb + GTm::k1 + t0, k1);
                ld(lb + GTm::k3 + t0, ka);
                ld(lb + GTm::k3 + kC + t0, kb);
                ld(lb + GTm::q2 + t0, qa);
                ld(lb + GTm::q2 + kC + t0, qb);
                ld(lb + GTm::k2 + t0, ea);
                ld(lb + GTm::k2 + kC + t0, eb);
                tmem_ld_wait();
                if (x0 == 8) arrive(&bar->acc_free);
#pragma unroll
                for (int y = 0; y < 8; y += 4) {
                    const float4 ga = ld_f4(rec + kGam + t0 + y), bg = ld_f4(rec + kBg + t0 + y),
                                 tb = ld_f4(rec + kTb + t0 + y);
                    const float gav[4] = {ga.x, ga.y, ga.z, ga.w}, bgv[4] = {bg.x, bg.y, bg.z, bg.w},
                                tbv[4] = {tb.x, tb.y, tb.z, tb.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int x = y + e;
                        const float dqi = gav[e] * __uint_as_float(q1[x]);
                        const float dki = bgv[e] * __uint_as_float(k1[x]);
                        const float dko = tbv[e] * (__uint_as_float(ka[x]) + __uint_as_float(kb[x]));
                        const float dqv = dqi + (__uint_as_float(qa[x]) + __uint_as_float(qb[x]));
                        const float dkv = (dki + dko) + (__uint_as_float(ea[x]) + __uint_as_float(eb[x]));
                        float s = 0.f;
                        if (r < D) {
                            const float qv = col_get(qc, x0 + x), kv = col_get(kc, x0 + x), o = kv * dko;
                            s = fmaf(qv, dqi, fmaf(kv, dki, -o));
                            outs += o;
                            if (e & 1) {
                                col_put2(sq, x0 + x - 1, dq_even, dqv);
                                col_put2(sk, x0 + x - 1, dk_even, dkv);
                            }
                            dq_even = dqv;
                            dk_even = dkv;
                        }
                        tok[x0 + x] = s;
                    }
                }
            }
            const float ts = reduce16(tok, lane);
            if ((lane & 1) == 0) part[L::pTok + q4 * kC + col0 + (lane >> 1)] = ts;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                outs += __shfl_xor_sync(0xffffffffu, outs, o);
                kept += __shfl_xor_sync(0xffffffffu, kept, o);
            }
            if (lane == 0) {
                part[L::pSum + (warp - 2)] = outs;
                part[L::pSum + kWarps + (warp - 2)] = kept;
            }
            fence_proxy_async_smem();
            named_barrier(1, 32 * kWarps);
            if (ct == 0) {
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
                    if (64 * b >= Dk) continue;
                    tma_store_3d(&tm_dq, base + L::out + b * kBlk, 64 * b, c0, bh);
                    tma_store_3d(&tm_dk, base + L::out + (D / 64 + b) * kBlk, 64 * b, c0, bh);
                }
                bulk_commit();
            }
            if (warp == 3) {  // dg: the reverse cumulative sum, two positions to a lane (fp32: the terms carry bf16 roundings)
                float v[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 2 * lane + e;
                    float a = 0.f;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        a += (part[L::pRow + y * 128 + j] + part[L::pRow + y * 128 + kC + j]) +
                             (part[L::pCol + y * kC + j] + part[L::pTok + y * kC + j]);
                    v[e] = a;
                }
                float tail = part[L::pSum + kWarps + (lane & (kWarps - 1))], os = part[L::pSum + (lane & (kWarps - 1))];
#pragma unroll
                for (int o = kWarps / 2; o > 0; o >>= 1) {
                    tail += __shfl_xor_sync(0xffffffffu, tail, o);
                    os += __shfl_xor_sync(0xffffffffu, os, o);
                }
                const float all = fmaf(tail, rec[kGam + kC - 1], os);
                const float both = v[0] + v[1];
                float run = both;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float x = __shfl_down_sync(0xffffffffu, run, o);
                    if (lane + o < 32) run += x;
                }
                const float after = run - both;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 2 * lane + e;
                    if (j >= n || !LA_DCHECK(c0 + j < N)) continue;
                    const size_t pos = (size_t)bh * N + c0 + j;
                    // a reset is where the count of resets goes up
                    const bool reset = rec[kSeg + j] != (j > 0 ? rec[kSeg + j - 1] : 0.f);
                    dg[pos] = __float2bfloat16_rn(reset ? 0.f : after + (e ? v[1] : both) + all);
                    dbeta[pos] = __float2bfloat16_rn(part[L::dBeta + j]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->b_free);  // this warp is done with Q, K and the gates
        }
        if (ct == 0) bulk_wait_all();
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool kSums>
cudaError_t sweeps(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                   const CUtensorMap& tdv, const StateArgs& sa, const ReverseArgs& ra, dim3 grid, int* err, cudaStream_t st) {
    GD_TRY(allow_smem(tc_gd_sweeps<D, kSums>, SweepSmem<D, kSums>::bytes));
    const char* name = kSums ? "tc_gd_sweep_sums" : "tc_gd_sweeps";
    launch_begin(name, st);
    const cudaError_t e = launch_pdl(tc_gd_sweeps<D, kSums>, grid, dim3(kThreads), SweepSmem<D, kSums>::bytes, st, tq, tk, tv,
                                     tdo, tdv, sa, ra, err);
    const cudaError_t e2 = launch_end(name, st);
    return e != cudaSuccess ? e : e2;
}

template <int D>
cudaError_t bwd(const BwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    const int BH = s.B * s.H, M = (s.N + kC - 1) / kC;
    CUtensorMap tq, tk, tv, tdo, tdq, tdk, tdv;
    if (!make_tmap_bf16_rows(&tq, a.q, BH, s.N, s.Dk, kC) || !make_tmap_bf16_rows(&tk, a.k, BH, s.N, s.Dk, kC) ||
        !make_tmap_bf16_rows(&tv, a.v, BH, s.N, s.Dv, kC) || !make_tmap_bf16_rows(&tdo, a.dout, BH, s.N, s.Dv, kC) ||
        !make_tmap_bf16_rows(&tdq, a.dq, BH, s.N, s.Dk, kC) || !make_tmap_bf16_rows(&tdk, a.dk, BH, s.N, s.Dk, kC) ||
        !make_tmap_bf16_rows(&tdv, a.dv, BH, s.N, s.Dv, kC))
        return cudaErrorInvalidValue;
    int* err = device_error_word();
    const Layout L = layout(s, true);
    float* recs = (float*)(ws + L.rec);
    uint8_t *mats = (uint8_t*)(ws + L.t), *X = (uint8_t*)(ws + L.X), *Y = (uint8_t*)(ws + L.Y), *S = (uint8_t*)(ws + L.S),
            *dS = (uint8_t*)(ws + L.dS);
    GD_TRY(prepare<D>(tq, tk, a.g, a.beta, recs, mats, s, M, true, err, st));
    StateArgs sa{};
    sa.recs = recs;
    sa.mats = mats;
    sa.mat_bytes = kMatsBwd;
    sa.x_tiles = X;
    sa.s_tiles = S;
    sa.M = M;
    sa.P = L.segs;
    sa.cps = L.cps;
    ReverseArgs ra{};
    ra.recs = recs;
    ra.mats = mats;
    ra.y_tiles = Y;
    ra.ds_tiles = dS;
    ra.M = M;
    ra.P = L.segs;
    ra.cps = L.cps;
    ra.Dk = ra.ek = s.Dk;
    ra.Dv = ra.ev = s.Dv;
    ra.segdS = a.dS;
    ra.dS0 = a.dS0;
    sa.S0 = a.S0;
    sa.dk = s.Dk;
    sa.dv = s.Dv;
    if (L.segs > 1) {
        sa.segB = (float*)(ws + L.segB);
        sa.segM = (float*)(ws + L.segM);
        ra.segB2 = (float*)(ws + L.segB2);
        GD_TRY((sweeps<D, true>(tq, tk, tv, tdo, tdv, sa, ra, dim3(L.segs, BH, D == 128 ? 3 : 2), err, st)));
        GD_TRY(join<D>(sa.segB, sa.segM, a.S0, (float*)(ws + L.segS), ra.segB2, a.dS, (float*)(ws + L.segdS), BH, L.segs,
                       s.Dk, s.Dv, err, st));
        sa.S0 = (float*)(ws + L.segS);
        sa.dk = sa.dv = D;
        ra.segdS = (float*)(ws + L.segdS);
        ra.ek = ra.ev = D;
    }
    GD_TRY((sweeps<D, false>(tq, tk, tv, tdo, tdv, sa, ra, dim3(L.segs, BH, 2), err, st)));
    GD_TRY(allow_smem(tc_gd_grads<D>, GradSmem<D>::bytes));
    launch_begin("tc_gd_grads", st);
    const int total = BH * M;
    const cudaError_t e =
        launch_pdl(tc_gd_grads<D>, dim3(total < 152 ? total : 152), dim3(kThreads), GradSmem<D>::bytes, st, tq, tk, tdo, tdq,
                   tdk, (const float*)recs, (const uint8_t*)X, (const uint8_t*)Y, (const uint8_t*)S, (const uint8_t*)dS,
                   (__nv_bfloat16*)a.dg, (__nv_bfloat16*)a.dbeta, s.N, M, total, s.Dk, err);
    const cudaError_t e2 = launch_end("tc_gd_grads", st);
    return e != cudaSuccess ? e : e2;
}

}  // namespace

cudaError_t tc_bwd(const BwdArgs& a, const la_shape& s, char* ws, cudaStream_t st) {
    return tc_dim(s) == 128 ? bwd<128>(a, s, ws, st) : bwd<64>(a, s, ws, st);
}

}  // namespace gd
}  // namespace la
