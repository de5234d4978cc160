// tc_gated_delta_states.cuh -- the block that carries a segment's state through its chunks, for the kernels of
// tc_gated_delta.cu (outputs, sums of segments) and tc_gated_delta_bwd.cu (what the gradient keeps).
#pragma once
#include "tc_gated_delta.cuh"

namespace la {
namespace gd {
namespace tcgd {
using namespace sm100;

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

// The block of segment p of head bh; map (kSum, D = 128): it forms the segment's map instead of its sum (with D = 64 the
// upper lanes, which have no value columns, carry the map).
template <int D, int kMode>
__device__ __forceinline__ void states_block(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                             const StateArgs& a, int p, int bh, bool map, int* err) {
    using L = FwdSmem<D, kMode>;
    using T = Tm<D>;
    constexpr int kSc = D / kHs;  // state columns of a thread
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars* bar = reinterpret_cast<Bars*>(base + L::bars);
    uint32_t* slot = reinterpret_cast<uint32_t*>(base + L::slot);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int M = a.M, cbeg = p * a.cps, nloc = min(M, cbeg + a.cps) - cbeg;
    LA_DCHECK(nloc >= 1);
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
            auto put = [&](int stride) {
#pragma unroll
                for (int x = 0; x < kTok; ++x)
                    if (x < n && LA_DCHECK(t0 + x < a.N)) o[x * stride] = __float2bfloat16_rn(__uint_as_float(w[x]) + __uint_as_float(w2[x]));
            };
            if (a.Dv == D) {
                if (r < D) put(D);  // a constant, for immediate offsets
            } else if (r < a.Dv) {
                put(a.Dv);
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
                    LA_DCHECK(cbeg + i < M && bh < (int)gridDim.y);
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
            LA_DCHECK(p < a.P && bh < (int)gridDim.y);
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
                if (c < a.Dk && LA_DCHECK(bh < (int)gridDim.y)) a.S_out[((size_t)bh * a.Dk + c) * a.Dv + r] = x & 1 ? S[x / 2].y : S[x / 2].x;
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

}  // namespace tcgd
}  // namespace gd
}  // namespace la
