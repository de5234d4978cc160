// tc_cross_bwd.cu -- tensor-core kernels of the gradient of cross attention.
//
//   cross_query_tc  Y = dO S^T, t = phi(q) . Y / den, dq = (Y / den - t / den z) phi'(q)
//                   R += X^T dO, r -= X^T t with X = phi(Q) / den          outputs, records of (R, r)
//   cross_key_tc    dk = (V R^T + r) phi'(k), dv = phi(K) R                outputs
//
// t needs no product of its own: dO . (phi(q) S) is phi(q) . (S dO), the row sum that the epilogue of Y forms.  dO and V enter
// their products as they land, without a pass over them.  dq is a small difference of large terms (the keys' weights vary
// little), so S enters as two bf16 parts and everything else of dq is fp32; dk keeps a rounding of X's and R's whole size, so R
// is two parts, and X as well.  Bound by memory: a chunk of 128 rows, 128 wide, is 96 KB (query) or 128 KB (key), 2.2 and 2.9 us
// of an SM's share of the copy rate, against 2 and 1.4 us for its products.  Two groups of four warps take alternate
// chunks, a thread a row; outputs go back into the stage's tiles for their store.
#include <cudaTypedefs.h>

#include "norm_common.cuh"
#include "tc_cross.cuh"

namespace la {
namespace cross {
namespace {

using norm::both;
using norm::fma2;
using norm::mul2;
using norm::Pairs;
using tc::bf_hi;
using tc::bf_lo;

constexpr int kThreads = 352;  // warp 0 TMA loads, 1 MMA, 2-9 two compute groups, 10 TMA stores
constexpr int T = 16384;       // 128 rows of a block

// A warpgroup gives registers back, or takes them, down or up to n a thread.
template <int n>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n)); }
template <int n>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n)); }

// A row of a tile through f(first column, its 16 bytes as 4 words): f may change the words.
template <int B, typename F>
__device__ __forceinline__ void row_words(const uint8_t* tile, int r, F f) {
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int lc = 0; lc < 8; ++lc) {
            const uint4 x = *reinterpret_cast<const uint4*>(tile + b * T + swz(r, lc));
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
            f(b, lc, u);
        }
}

// ------------------------------------------------------------------ query pass
// A stage holds Q (then X's hi part, then dq) and dO.  X's lo part: for KB = 1 in the stage, the second 64-row half of one
// 128-row product; for KB = 2 in a tile of its own, for which shared memory has no second.  t enters as the first two columns
// (hi and lo) of a 16-column operand W, K-major, of whose rows only 8 are held: rows 8-15 of a block are read from the 1 KB
// behind it (the other block's rows, or z and the barriers) and make columns of the result that nothing reads.
//
// The compute warps hold their row's phi in fp32 throughout (128 registers), which they get from the other warpgroup:
// 384 threads of 168 registers are 128 of 80 and 256 of 208.  A chunk's phases, each overlapping the other group's:
//   phi, den, X -> X^T dO may start;   Y -> t -> X^T t may start;   Y -> dq, which waits for X's tile.
constexpr int kQueryThreads = 384;  // warp 0 TMA loads, 1 MMA, 2 TMA stores, 4-11 two compute groups

template <int KB, int VB>
struct QuerySmem {
    static constexpr int kLo = KB == 1 ? T : 0, kDo = (KB == 1 ? 2 : KB) * T, kStage = kDo + VB * T;
    static constexpr int kS = 2 * (int)image_part(KB, VB), kX = KB == 2 ? KB * T : 0;
    static constexpr int kStages = (229376 - kS - kX) / kStage > 4 ? 4 : (229376 - kS - kX) / kStage;
    static constexpr int S0 = kStages * kStage, X0 = S0 + kS;
    static constexpr int W = X0 + kX;          // 2 blocks of 8 rows x 128 bytes
    static constexpr int z0 = W + 2048;        // float[64 KB]
    static constexpr int bars = z0 + 512;
    static constexpr int total = bars + 512;   // W's last read ends here
    static_assert(kStages >= 2 && total <= 232448, "query pass: shared memory");
};

template <int KB, int VB>
__global__ void __launch_bounds__(kQueryThreads, 1)
cross_query_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
               const __grid_constant__ CUtensorMap tm_dq, const char* __restrict__ image, float* __restrict__ rec, Rows rows, int Dk,
               int slots, int* err) {
    using SM = QuerySmem<KB, VB>;
    constexpr int NS = SM::kStages;
    constexpr uint32_t kY = 0, kR = 128 * KB, kW = kR + 64 * VB;  // TMEM: two Y, R, the columns of r
    constexpr uint32_t kCols = kW + 16 <= 256 ? 256 : 512;
    extern __shared__ __align__(1024) uint8_t smem[];
    struct Bars {
        uint64_t full[4], empty[4], staged[4], s_full, s_empty, y_done[2], y_free[2], x_ready[2], w_ready[2], r_done[2], x_free, r_flushed,
            final_mma;
        uint32_t tmem;
        Span span;
    };
    static_assert(sizeof(Bars) <= 512, "barriers");
    Bars* bar = reinterpret_cast<Bars*>(smem + SM::bars);
    const float* zs = reinterpret_cast<const float*>(smem + SM::z0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    LA_DCHECK((smem_u32(smem) & 1023) == 0);
    if (tid == 32) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 1);
            mbar_init(&bar->staged[s], 128);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bar->y_done[g], 1);
            mbar_init(&bar->y_free[g], 128);
            mbar_init(&bar->x_ready[g], 128);
            mbar_init(&bar->w_ready[g], 128);
            mbar_init(&bar->r_done[g], 1);
        }
        mbar_init(&bar->s_full, 1);
        mbar_init(&bar->s_empty, 9);  // the products and the eight compute warps (z)
        mbar_init(&bar->x_free, 1);
        mbar_init(&bar->r_flushed, 128);
        mbar_init(&bar->final_mma, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_do);
        tma_prefetch_desc(&tm_dq);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(&bar->tmem, kCols);
        tmem_relinquish();
    }
    for (int x = tid; x < 2048 / 16; x += kQueryThreads) reinterpret_cast<uint4*>(smem + SM::W)[x] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    pdl_enter();  // launched with programmatic dependent launch
    if (warp == 0) {
        const Span sp = span_of(rows, kRowChunk, false, blockIdx.x, gridDim.x);
        if (lane == 0) bar->span = sp;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;
    Walk w(rows, kRowChunk, bar->span);

    if (warp < 4) reg_dec<80>();
    if (warp == 0) {
        if (lane == 0) {
            int i = 0, heads = 0;
            bool first = true;
            for (; w.more(); w.next(), ++i) {
                const int s = i % NS;
                if (!mbar_wait(&bar->empty[s], ((i / NS) & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                uint8_t* st = smem + s * SM::kStage;
                mbar_arrive_expect_tx(&bar->full[s], (KB + VB) * T);
                check_copy(0, w.row0(), rows.M, w.bh, rows.heads());
                for (int b = 0; b < VB; ++b) tma_load_3d(st + SM::kDo + b * T, &tm_do, 64 * b, w.row0(), w.bh, &bar->full[s]);
                for (int b = 0; b < KB; ++b) tma_load_3d(st + b * T, &tm_q, 64 * b, w.row0(), w.bh, &bar->full[s]);
                if (first) {  // after the chunk's own tiles: those need no wait for the head before
                    if (!mbar_wait(&bar->s_empty, (heads & 1) ^ 1, err, LA_ERR_TIMEOUT)) {
                        ++i;
                        break;
                    }
                    const char* im = image + (size_t)w.bh * image_bytes(KB, VB);
                    mbar_arrive_expect_tx(&bar->s_full, SM::kS + 256 * KB);
                    bulk_load(smem + SM::S0, im, SM::kS, &bar->s_full);
                    bulk_load(smem + SM::z0, im + SM::kS, 256 * KB, &bar->s_full);
                    ++heads;
                }
                first = w.last();
            }
            mbar_drain(bar->full, NS, i, err, LA_ERR_TIMEOUT);  // no copy is left in flight
            mbar_drain(&bar->s_full, 1, heads, err, LA_ERR_TIMEOUT);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t id_y = idesc_bf16_f32(128, 64 * KB, 0, 0), id_r = idesc_bf16_f32(128, 64 * VB, 1, 1),
                               id_w = idesc_bf16_f32(128, 16, 1, 0);
            const uint32_t aS = smem_u32(smem + SM::S0), aSl = aS + (uint32_t)image_part(KB, VB), aW = smem_u32(smem + SM::W),
                           aX = smem_u32(smem + SM::X0);
            bool ok = true, y_first = true, first = true, r_first = true;
            int yi = 0, ri = 0, heads = 0, flushes = 0;
            Walk wy = w;
            auto issue_y = [&]() {  // Y of chunk yi: dO is all it needs, so it runs a chunk ahead
                const int g = yi & 1, s = yi % NS;
                if (y_first) ok = ok && mbar_wait(&bar->s_full, heads++ & 1, err, LA_ERR_TIMEOUT);
                ok = ok && mbar_wait(&bar->full[s], (yi / NS) & 1, err, LA_ERR_TIMEOUT) &&
                     mbar_wait(&bar->y_free[g], ((yi >> 1) & 1) ^ 1, err, LA_ERR_TIMEOUT);
                if (!ok) return;
                tc_fence_after();
                const uint32_t aD = smem_u32(smem + s * SM::kStage + SM::kDo), acc = tmem + kY + 64 * KB * g;
#pragma unroll
                for (int kk = 0; kk < 4 * VB; ++kk) {
                    mma_ss(acc, desc_k(aD, kk, T), desc_k(aS, kk, 8192 * KB), id_y, kk > 0);
                    mma_ss(acc, desc_k(aD, kk, T), desc_k(aSl, kk, 8192 * KB), id_y, 1);
                }
                mma_commit(&bar->y_done[g]);
                y_first = wy.last();
                if (y_first) mma_commit(&bar->s_empty);
                wy.next();
                ++yi;
            };
            auto issue_r = [&]() {  // X^T t of chunk ri (of X's hi part for KB = 2: t is smaller than dO . v)
                const int g = ri & 1, s = ri % NS;
                ok = ok && mbar_wait(&bar->w_ready[g], (ri >> 1) & 1, err, LA_ERR_TIMEOUT);
                if (!ok) return;
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * SM::kStage);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) mma_ss(tmem + kW, desc_mn(st, kk, T), desc_k(aW, kk, 1024), id_w, !r_first || kk > 0);
                mma_commit(&bar->r_done[g]);
                r_first = false;
                ++ri;
            };
            for (int i = 0; w.more() && ok; w.next(), ++i) {
                const int g = i & 1, s = i % NS;
                while (ok && yi <= i) issue_y();
                ok = ok && mbar_wait(&bar->x_ready[g], (i >> 1) & 1, err, LA_ERR_TIMEOUT);
                if (first && flushes > 0) ok = ok && mbar_wait(&bar->r_flushed, (flushes - 1) & 1, err, LA_ERR_TIMEOUT);
                if (!ok) break;
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * SM::kStage), aD = st + SM::kDo;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    mma_ss(tmem + kR, desc_mn(st, kk, T), desc_mn(aD, kk, T), id_r, !first || kk > 0);
                    if (KB == 2) mma_ss(tmem + kR, desc_mn(aX, kk, T), desc_mn(aD, kk, T), id_r, 1);
                }
                mma_commit(&bar->x_free);
                first = w.last();
                while (ok && ri < (first ? i + 1 : i)) issue_r();  // a head's are all issued before the next head begins
                if (first) r_first = true, ++flushes;
                if (ok && wy.more() && yi == i + 1 && !y_first) issue_y();  // unless it needs the next head's S
            }
            mma_commit(&bar->final_mma);  // every product is complete before the accumulators are given back
            mbar_wait(&bar->final_mma, 0, err, LA_ERR_TIMEOUT);
        }
    } else if (warp == 2) {
        if (lane == 0) {  // stores: a stage is empty once its dq has been read
            for (int i = 0; w.more(); w.next(), ++i) {
                const int s = i % NS;
                if (!mbar_wait(&bar->staged[s], (i / NS) & 1, err, LA_ERR_TIMEOUT)) break;
                check_copy(0, w.row0(), rows.M, w.bh, rows.heads());
                for (int b = 0; b < KB; ++b) tma_store_3d(&tm_dq, smem + s * SM::kStage + b * T, 64 * b, w.row0(), w.bh);
                bulk_commit();
                bulk_wait_read_all();
                mbar_arrive(&bar->empty[s]);
            }
            bulk_wait_all();
        }
    } else if (warp >= 4) {
        reg_inc<208>();
        const int g = (warp - 4) >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, acc = tmem + kY + 64 * KB * g + lanes;
        int i = 0, heads = 0;
        bool first = true;
        for (; w.more(); w.next(), ++i) {
            if (first) ++heads;
            const bool last = first = w.last();
            if ((i & 1) == g) {
                const int s = i % NS;
                uint8_t* st = smem + s * SM::kStage;
                if (!warp_wait(&bar->s_full, (heads - 1) & 1, err) || !warp_wait(&bar->full[s], (i / NS) & 1, err)) break;
                // phi of the row, its normaliser, X (rows behind the last query and padded columns, which hold phi(0): 0)
                float2 p[32 * KB], s2 = both(0.f);
                row_words<KB>(st, r, [&](int b, int lc, const uint32_t(&u)[4]) {
                    float2 zv[4];
                    Pairs<float>::get(zs + 64 * b + 8 * lc, reinterpret_cast<float2(&)[2]>(zv[0]));
                    Pairs<float>::get(zs + 64 * b + 8 * lc + 4, reinterpret_cast<float2(&)[2]>(zv[2]));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = make_float2(phi_f(bf_lo(u[e])), phi_f(bf_hi(u[e])));
                        p[32 * b + 4 * lc + e] = f;
                        s2 = fma2(f, zv[e], s2);
                    }
                });
                const float inv = over(s2.x + s2.y), xi = r < w.rows() ? inv : 0.f;
                // KB = 2: the product that reads the lo tile of the chunk before is through
                if (KB == 2 && i > 0 && !warp_wait(&bar->x_free, (i - 1) & 1, err)) break;
                uint8_t* lo = KB == 2 ? smem + SM::X0 : st + SM::kLo;
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int lc = 0; lc < 8; ++lc) {
                        uint4 h, l;
                        uint32_t *hw = reinterpret_cast<uint32_t*>(&h), *lw = reinterpret_cast<uint32_t*>(&l);
                        const float2 k = both(64 * b + 8 * lc < Dk ? xi : 0.f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 x = mul2(p[32 * b + 4 * lc + e], k);
                            split2(x.x, x.y, hw[e], lw[e]);
                        }
                        *reinterpret_cast<uint4*>(st + b * T + swz(r, lc)) = h;
                        *reinterpret_cast<uint4*>(lo + b * T + swz(r, lc)) = l;
                    }
                fence_proxy_async_smem();
                mbar_arrive(&bar->x_ready[g]);
                // t = phi(q) . Y / den
                if (!warp_wait(&bar->y_done[g], (i >> 1) & 1, err)) break;
                tc_fence_after();
                s2 = both(0.f);
#pragma unroll
                for (int b = 0; b < 2 * KB; ++b) {
                    uint32_t y[32];
                    tmem_ld32(acc + 32 * b, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        s2 = fma2(p[16 * b + e], make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), s2);
                }
                const float t = (s2.x + s2.y) * inv;
                if (i > 0 && !warp_wait(&bar->r_done[(i - 1) & 1], ((i - 1) >> 1) & 1, err)) break;  // W is read
                {
                    uint32_t th, tl;
                    split2(-t, 0.f, th, tl);
                    uint8_t* at = smem + SM::W + (r >> 6) * 1024 + (r & 7) * 2;
                    const int lc = (r & 63) >> 3;  // rows 0 and 1 of the operand
                    *reinterpret_cast<uint16_t*>(at + swz(0, lc)) = (uint16_t)th;
                    *reinterpret_cast<uint16_t*>(at + swz(1, lc)) = (uint16_t)tl;
                }
                fence_proxy_async_smem();
                mbar_arrive(&bar->w_ready[g]);
                // dq, packed until the row's tile is free
                const float2 gz = both(-t * inv), iv = both(inv);
                uint32_t dq[32 * KB];
#pragma unroll
                for (int b = 0; b < 2 * KB; ++b) {
                    uint32_t y[32];
                    tmem_ld32(acc + 32 * b, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        float2 zv[2];
                        Pairs<float>::get(zs + 32 * b + 2 * e, zv);
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            const int c = 2 * (e + o);
                            const float2 f = p[16 * b + e + o];
                            const float2 d = mul2(fma2(gz, zv[o], mul2(iv, make_float2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])))),
                                                  make_float2(dphi_from_phi(f.x), dphi_from_phi(f.y)));
                            dq[16 * b + e + o] = pack_bf16x2(d.x, d.y);
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(&bar->y_free[g]);
                if (!warp_wait(&bar->r_done[g], (i >> 1) & 1, err)) break;
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int lc = 0; lc < 8; ++lc)
                        *reinterpret_cast<uint4*>(st + b * T + swz(r, lc)) =
                            make_uint4(dq[32 * b + 4 * lc], dq[32 * b + 4 * lc + 1], dq[32 * b + 4 * lc + 2], dq[32 * b + 4 * lc + 3]);
                fence_proxy_async_smem();
                mbar_arrive(&bar->staged[s]);
                if (last) {  // this head's sums
                    tc_fence_after();
                    if (LA_DCHECK((int)blockIdx.x + w.bh < slots)) {
                        float* out = rec + (size_t)(blockIdx.x + w.bh) * record_floats(VB);
                        tc::tmem_row_to_global<64 * VB>(tmem + kR + lanes, out + (size_t)r * 64 * VB);
                        uint32_t c[16];
                        tmem_ld16(tmem + kW + lanes, c);
                        tmem_ld_wait();
                        out[128 * 64 * VB + r] = __uint_as_float(c[0]) + __uint_as_float(c[1]);
                    }
                    tc_fence_before();
                    mbar_arrive(&bar->r_flushed);
                }
            }
            if (last) {  // z is no longer read
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->s_empty);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// ------------------------------------------------------------------ key pass
// A stage holds K (phi's bf16 copy in place) and V; then dv and, VB blocks on, dk.  V R^T starts as V lands, and its
// epilogue runs beside phi(K) R where dk's place is not K's (KB <= VB).  phi(K) enters dv's product rounded once: its
// errors are independent from column to column of R, whose entries are not.  phi'(k) is formed from k itself.
template <int KB, int VB>
struct KeySmem {
    static constexpr int kV = KB * T, kDk = VB * T, kStage = (KB + VB) * T, kR = 2 * (int)image_part(KB, VB);
    static constexpr int kStages = (229376 - kR) / kStage > 4 ? 4 : (229376 - kR) / kStage;
    static constexpr int R0 = kStages * kStage, r0 = R0 + kR, bars = r0 + 512, total = bars + 512;
    static_assert(kStages >= 2 && total <= 232448, "key pass: shared memory");
};

template <int KB, int VB>
__global__ void __launch_bounds__(kThreads, 1)
cross_key_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
             const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv, const char* __restrict__ image,
             Rows keys, int* err) {
    using SM = KeySmem<KB, VB>;
    constexpr int NS = SM::kStages;
    constexpr uint32_t kSet = 64 * (KB + VB);  // TMEM of a group: dK without r and phi', then dV
    constexpr uint32_t kCols = 2 * kSet <= 256 ? 256 : 512;
    extern __shared__ __align__(1024) uint8_t smem[];
    struct Bars {
        uint64_t full[4], empty[4], staged[4], s_full, s_empty, ready[2], k_done[2], v_done[2], acc_free[2], final_mma;
        uint32_t tmem;
        Span span;
    };
    static_assert(sizeof(Bars) <= 512, "barriers");
    Bars* bar = reinterpret_cast<Bars*>(smem + SM::bars);
    const float* rs = reinterpret_cast<const float*>(smem + SM::r0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    LA_DCHECK((smem_u32(smem) & 1023) == 0);
    if (tid == 32) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 1);
            mbar_init(&bar->staged[s], 128);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bar->ready[g], 128);
            mbar_init(&bar->k_done[g], 1);
            mbar_init(&bar->v_done[g], 1);
            mbar_init(&bar->acc_free[g], 128);
        }
        mbar_init(&bar->s_full, 1);
        mbar_init(&bar->s_empty, 9);  // the products and the eight compute warps (r)
        mbar_init(&bar->final_mma, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_dk);
        tma_prefetch_desc(&tm_dv);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(&bar->tmem, kCols);
        tmem_relinquish();
    }
    pdl_enter();  // launched with programmatic dependent launch
    if (warp == 0) {
        const Span sp = span_of(keys, kRowChunk, false, blockIdx.x, gridDim.x);
        if (lane == 0) bar->span = sp;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;
    Walk w(keys, kRowChunk, bar->span);

    if (warp == 0) {
        if (lane == 0) {
            int i = 0, heads = 0;
            bool first = true;
            for (; w.more(); w.next(), ++i) {
                const int s = i % NS;
                if (!mbar_wait(&bar->empty[s], ((i / NS) & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                uint8_t* st = smem + s * SM::kStage;
                mbar_arrive_expect_tx(&bar->full[s], (KB + VB) * T);
                check_copy(0, w.row0(), keys.M, w.bh, keys.heads());
                for (int b = 0; b < KB; ++b) tma_load_3d(st + b * T, &tm_k, 64 * b, w.row0(), w.bh, &bar->full[s]);
                for (int b = 0; b < VB; ++b) tma_load_3d(st + SM::kV + b * T, &tm_v, 64 * b, w.row0(), w.bh, &bar->full[s]);
                if (first) {  // after the chunk's own tiles: those need no wait for the head before
                    if (!mbar_wait(&bar->s_empty, (heads & 1) ^ 1, err, LA_ERR_TIMEOUT)) {
                        ++i;
                        break;
                    }
                    const char* im = image + (size_t)w.bh * image_bytes(KB, VB);
                    mbar_arrive_expect_tx(&bar->s_full, SM::kR + 256 * KB);
                    bulk_load(smem + SM::R0, im, SM::kR, &bar->s_full);
                    bulk_load(smem + SM::r0, im + SM::kR, 256 * KB, &bar->s_full);
                    ++heads;
                }
                first = w.last();
            }
            mbar_drain(bar->full, NS, i, err, LA_ERR_TIMEOUT);  // no copy is left in flight
            mbar_drain(&bar->s_full, 1, heads, err, LA_ERR_TIMEOUT);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t id_k = idesc_bf16_f32(128, 64 * KB, 0, 0), id_v = idesc_bf16_f32(128, 64 * VB, 0, 1);
            const uint32_t aR = smem_u32(smem + SM::R0), aRl = aR + (uint32_t)image_part(KB, VB);
            int i = 0, vi = 0, heads = 0;
            Walk wv = w;  // V R^T runs a chunk ahead
            bool v_first = true, ok = true;
            auto issue_k = [&]() {  // dK without r and phi' of chunk vi
                const int g = vi & 1, s = vi % NS;
                if (v_first) ok = ok && mbar_wait(&bar->s_full, heads++ & 1, err, LA_ERR_TIMEOUT);
                ok = ok && mbar_wait(&bar->full[s], (vi / NS) & 1, err, LA_ERR_TIMEOUT) &&
                     mbar_wait(&bar->acc_free[g], ((vi >> 1) & 1) ^ 1, err, LA_ERR_TIMEOUT);
                if (!ok) return;
                tc_fence_after();
                const uint32_t aV = smem_u32(smem + s * SM::kStage + SM::kV), acc = tmem + kSet * g;
#pragma unroll
                for (int kk = 0; kk < 4 * VB; ++kk) {
                    mma_ss(acc, desc_k(aV, kk, T), desc_k(aR, kk, 8192 * KB), id_k, kk > 0);
                    mma_ss(acc, desc_k(aV, kk, T), desc_k(aRl, kk, 8192 * KB), id_k, 1);
                }
                mma_commit(&bar->k_done[g]);
                v_first = wv.last();
                wv.next();
                ++vi;
            };
            for (; w.more() && ok; w.next(), ++i) {
                const int g = i & 1, s = i % NS;
                while (ok && vi <= i) issue_k();
                if (!ok || !mbar_wait(&bar->ready[g], (i >> 1) & 1, err, LA_ERR_TIMEOUT)) break;
                tc_fence_after();
                const uint32_t aK = smem_u32(smem + s * SM::kStage), acc = tmem + kSet * g + 64 * KB;
#pragma unroll
                for (int kk = 0; kk < 4 * KB; ++kk) {
                    mma_ss(acc, desc_k(aK, kk, T), desc_mn(aR, kk, 8192 * KB), id_v, kk > 0);
                    mma_ss(acc, desc_k(aK, kk, T), desc_mn(aRl, kk, 8192 * KB), id_v, 1);
                }
                mma_commit(&bar->v_done[g]);
                if (w.last()) mma_commit(&bar->s_empty);
                // the next chunk's, unless it needs the next head's R, for which this head has to be through
                if (wv.more() && vi == i + 1 && !v_first) issue_k();
            }
            mma_commit(&bar->final_mma);  // every product is complete before the accumulators are given back
            mbar_wait(&bar->final_mma, 0, err, LA_ERR_TIMEOUT);
        }
    } else if (warp < 10) {
        const int g = (warp - 2) >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t acc = tmem + kSet * g + ((uint32_t)(32 * (warp & 3)) << 16);
        int i = 0, heads = 0;
        bool first = true;
        for (; w.more(); w.next(), ++i) {
            if (first) ++heads;
            const bool last = first = w.last();
            if ((i & 1) == g) {
                const int s = i % NS;
                const bool live = r < w.rows();
                uint8_t* st = smem + s * SM::kStage;
                if (!warp_wait(&bar->s_full, (heads - 1) & 1, err) || !warp_wait(&bar->full[s], (i / NS) & 1, err)) break;
                uint32_t k[32 * KB];
                row_words<KB>(st, r, [&](int b, int lc, const uint32_t(&u)[4]) {
                    uint4 x;
                    uint32_t* p = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        k[32 * b + 4 * lc + e] = u[e];
                        p[e] = pack_bf16x2(phi_f(bf_lo(u[e])), phi_f(bf_hi(u[e])));
                    }
                    *reinterpret_cast<uint4*>(st + b * T + swz(r, lc)) = x;
                });
                fence_proxy_async_smem();
                mbar_arrive(&bar->ready[g]);
                if (KB > VB && !warp_wait(&bar->v_done[g], (i >> 1) & 1, err)) break;  // dk lies over phi(K)
                if (!warp_wait(&bar->k_done[g], (i >> 1) & 1, err)) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 2 * KB; ++b) {
                    uint32_t y[32];
                    tmem_ld32(acc + 32 * b, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 x;
                        uint32_t* o = reinterpret_cast<uint32_t*>(&x);
                        const float4 ra = *reinterpret_cast<const float4*>(rs + 32 * b + 8 * c);
                        const float4 rb = *reinterpret_cast<const float4*>(rs + 32 * b + 8 * c + 4);
                        const float rr[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t kw = k[16 * b + 4 * c + e];
                            const float s0 = ex2_approx(fminf(bf_lo(kw), 0.f) * 1.4426950408889634f);
                            const float s1 = ex2_approx(fminf(bf_hi(kw), 0.f) * 1.4426950408889634f);
                            o[e] = pack_bf16x2((__uint_as_float(y[8 * c + 2 * e]) + rr[2 * e]) * s0,
                                               (__uint_as_float(y[8 * c + 2 * e + 1]) + rr[2 * e + 1]) * s1);
                        }
                        if (!live) x = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(st + SM::kDk + (b >> 1) * T + swz(r, 4 * (b & 1) + c)) = x;
                    }
                }
                if (KB <= VB && !warp_wait(&bar->v_done[g], (i >> 1) & 1, err)) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 2 * VB; ++b) {
                    uint32_t y[32];
                    tmem_ld32(acc + 64 * KB + 32 * b, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 x;
                        uint32_t* o = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = pack_bf16x2(__uint_as_float(y[8 * c + 2 * e]), __uint_as_float(y[8 * c + 2 * e + 1]));
                        if (!live) x = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(st + (b >> 1) * T + swz(r, 4 * (b & 1) + c)) = x;
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&bar->acc_free[g]);
                mbar_arrive(&bar->staged[s]);
            }
            if (last) {  // r is no longer read
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->s_empty);
            }
        }
    } else if (lane == 0) {
        // stores: a stage is empty once its outputs have been read
        for (int i = 0; w.more(); w.next(), ++i) {
            const int s = i % NS;
            if (!mbar_wait(&bar->staged[s], (i / NS) & 1, err, LA_ERR_TIMEOUT)) break;
            const uint8_t* st = smem + s * SM::kStage;
            check_copy(0, w.row0(), keys.M, w.bh, keys.heads());
            for (int b = 0; b < KB; ++b) tma_store_3d(&tm_dk, st + SM::kDk + b * T, 64 * b, w.row0(), w.bh);
            for (int b = 0; b < VB; ++b) tma_store_3d(&tm_dv, st + b * T, 64 * b, w.row0(), w.bh);
            bulk_commit();
            bulk_wait_read_all();
            mbar_arrive(&bar->empty[s]);
        }
        bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

}  // namespace

cudaError_t tc_bwd(const BwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st) {
    const TcLayout l = tc_layout(s, LA_OP_CROSS_BWD);
    const Rows keys = key_rows(s, a.lens), rows = grouped_queries(s);
    float* rec = reinterpret_cast<float*>(ws);
    if (a.S) {
        CR_TRY(tc_join(nullptr, a.S, a.z, ws + l.S, nullptr, nullptr, keys, kSumRows, 1, s, st));
    } else {
        CR_TRY(tc_sums(a.k, a.v, keys, rec, l.sum_ctas, s, st));
        CR_TRY(tc_join(rec, nullptr, nullptr, ws + l.S, nullptr, nullptr, keys, kSumRows, l.sum_ctas, s, st));
    }
    CUtensorMap tq, td, tdq, tk, tv, tdk, tdv;
    if (!make_tmap_bf16_rows(&tq, a.q, rows.heads(), rows.M, s.Dk, kRowChunk) ||
        !make_tmap_bf16_rows(&td, a.dout, rows.heads(), rows.M, s.Dv, kRowChunk) ||
        !make_tmap_bf16_rows(&tdq, a.dq, rows.heads(), rows.M, s.Dk, kRowChunk) ||
        !make_tmap_bf16_rows(&tk, a.k, keys.heads(), keys.M, s.Dk, kRowChunk) ||
        !make_tmap_bf16_rows(&tv, a.v, keys.heads(), keys.M, s.Dv, kRowChunk) ||
        !make_tmap_bf16_rows(&tdk, a.dk, keys.heads(), keys.M, s.Dk, kRowChunk) ||
        !make_tmap_bf16_rows(&tdv, a.dv, keys.heads(), keys.M, s.Dv, kRowChunk))
        return cudaErrorInvalidValue;
    int* err = device_error_word();
    auto go = [&](auto query, size_t qs, auto key, size_t ks) {
        CR_TRY(tc_run("cross_query_tc", query, dim3(l.query_ctas), kQueryThreads, qs, st, tq, td, tdq, (const char*)ws + l.S, rec, rows,
                      s.Dk, l.query_ctas + rows.heads(), err));
        CR_TRY(tc_join(rec, nullptr, nullptr, ws + l.R, nullptr, nullptr, rows, kRowChunk, l.query_ctas, s, st));
        return tc_run("cross_key_tc", key, dim3(l.key_ctas), kThreads, ks, st, tk, tv, tdk, tdv, (const char*)ws + l.R, keys, err);
    };
    cudaError_t e;
    switch (2 * blocks64(s.Dk) + blocks64(s.Dv)) {
        case 3: e = go(cross_query_tc<1, 1>, QuerySmem<1, 1>::total, cross_key_tc<1, 1>, KeySmem<1, 1>::total); break;
        case 4: e = go(cross_query_tc<1, 2>, QuerySmem<1, 2>::total, cross_key_tc<1, 2>, KeySmem<1, 2>::total); break;
        case 5: e = go(cross_query_tc<2, 1>, QuerySmem<2, 1>::total, cross_key_tc<2, 1>, KeySmem<2, 1>::total); break;
        default: e = go(cross_query_tc<2, 2>, QuerySmem<2, 2>::total, cross_key_tc<2, 2>, KeySmem<2, 2>::total); break;
    }
    if (e != cudaSuccess || !a.lens) return e;
    return clear_behind(a.dk, a.dv, keys, s, st);
}

}  // namespace cross
}  // namespace la
