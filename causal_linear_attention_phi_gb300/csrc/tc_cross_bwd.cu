// tc_cross_bwd.cu -- tensor-core kernels of the gradient of cross attention.
//
//   cross_query_tc  Y = dO S^T, t = phi(q) . Y / den, dq = (Y / den - t / den z) phi'(q)
//                   R += X^T dO, r -= X^T t with X = phi(Q) / den          outputs, records of (R, r)
//   cross_key_tc    dk = (V R^T + r) phi'(k), dv = phi(K) R                outputs
//
// t needs no product of its own: dO . (phi(q) S) is phi(q) . (S dO), the row sum that the epilogue of Y forms.  dO and V enter
// their products as they land, without a pass over them.  dq is a small difference of large terms (the keys' weights vary
// little), so S enters centred (cross_join_tc; t, r and Y are those of the centred S) and as two bf16 parts, and everything else
// of dq is fp32; dk keeps a rounding of X's and of R's whole size: R is two parts, X one (see below).  Bound by memory, then by what passes through shared memory: a chunk of 128 rows, 128
// wide, is 96 KB (query) or 128 KB (key), 2.2 and 2.9 us of an SM's share of the copy rate, and its products, copies and
// epilogues move four times that between shared memory and the rest.  Two groups of eight warps take alternate chunks, half
// a row to a thread.  Measured at B=2 H=16 N=M=32768 128 x 128: query pass 161 us (0.74 of the copy rate), key pass 168 (0.94).
#include <cudaTypedefs.h>

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

constexpr int T = 16384;       // 128 rows of a block

// A warpgroup gives registers back, or takes them, down or up to n a thread.
template <int n>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n)); }
template <int n>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n)); }

// Wait until all but this thread's last committed store have finished reading shared memory.
__device__ __forceinline__ void bulk_wait_read_all_but_one() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

// A float of each lane to a column of tensor memory, for another warp of the same lanes to read after a barrier.
__device__ __forceinline__ void tmem_put(uint32_t taddr, float x) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(x)) : "memory");
    tmem_st_wait();
    tc_fence_before();
}
// The sum of two neighbouring columns.
__device__ __forceinline__ float tmem_sum2(uint32_t taddr) {
    uint32_t a, b;
    tc_fence_after();
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(taddr));
    tmem_ld_wait();
    return __uint_as_float(a) + __uint_as_float(b);
}

// Whether v holds for both warps of a pair (barrier `id`, 64 threads); what either wrote to shared memory is then seen by both.
__device__ __forceinline__ bool pair_all(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id)
        : "memory");
    return r != 0;
}

// ------------------------------------------------------------------ query pass
// A stage holds Q (then X) and dO; dq has a tile of its own, so a stage is free as soon as its products are through.  X is rounded
// once for KB = 2: dk is then 1.4 times as far off as its own rounding makes it (a second part would double the product
// and its reads of shared memory, which is what bounds this kernel: 280 us instead of 190 at B=2 H=16 N=32768).  For KB = 1 a lo part fills the
// second 64-row half of the 128-row product for nothing.  t enters as the first two columns
// (hi and lo) of a 16-column operand W, K-major, of whose rows only 8 are held: rows 8-15 of a block are read from the 1 KB
// behind it (the other block's rows, or z and the barriers) and make columns of the result that nothing reads.
//
// R and r stay in tensor memory for kPeriod chunks of a head only, as additions there are cut off (cross_sums_tc): then they are
// added to the block's record of the head, in fp32 and rounded to nearest.  No registers are free for them; the record is in L2.
// (131,072 queries in one accumulator: dk and dv 7e-4 short.  B=2 H=16 Hk=4 N=65536 M=131071 128 x 128: 497 us with a period of 32
// chunks, 473 of 64, 464 without one; B=2 H=16 N=32768: 351, 337, 337.)
//
// Two groups of eight warps; a thread holds half a row's phi in fp32 throughout, and the two threads of a row join their parts of
// den and of t through tensor memory, shared memory being full (a whole row to a thread took 343 us where this took 264:
// twice the code, of which the instruction cache held half, and two warps to a scheduler).  Registers come from the other
// warpgroup: 640 threads of 96 are 128 of 56 and 512 of 104.  A chunk's phases, each overlapping the other group's:
//   phi, den, X -> X^T dO may start;   Y -> t -> X^T t may start;   Y -> dq.
constexpr int kQueryThreads = 640;  // warp 0 TMA loads, 1 MMA of Y and R, 2 TMA stores, 3 MMA of r, 4-19 two compute groups
constexpr int kPeriod = 64;

// A walk's periods: where the accumulators of R and r are closed, the last chunk of a head or kPeriod chunks of it.
struct Period {
    int in = 0;  // chunks of the period so far
    __device__ bool close(const Walk& w) {  // whether chunk w ends its period; once for each chunk, in turn
        const bool c = w.last() || ++in == kPeriod;
        if (c) in = 0;
        return c;
    }
};

// kCols fp32 columns of a row from tensor memory, written to the row of a record or added to it.
template <int kCols>
__device__ __forceinline__ void tmem_row_to_record(uint32_t taddr, float* dst, bool add) {
#pragma unroll
    for (int b = 0; b < kCols / 16; ++b) {
        uint32_t w[16];
        tmem_ld16(taddr + 16 * b, w);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 16; x += 4) {
            float4* to = reinterpret_cast<float4*>(dst + 16 * b + x);
            float4 f = make_float4(__uint_as_float(w[x]), __uint_as_float(w[x + 1]), __uint_as_float(w[x + 2]), __uint_as_float(w[x + 3]));
            if (add) {
                const float4 was = *to;
                f.x += was.x, f.y += was.y, f.z += was.z, f.w += was.w;
            }
            *to = f;
        }
    }
}

template <int KB, int VB>
struct QuerySmem {
    static constexpr int kLo = T, kDo = 2 * T, kStage = kDo + VB * T;  // Q: two blocks, or X's parts
    static constexpr int kS = 2 * (int)image_part(KB, VB), kOut = KB * T;
    static constexpr int kStages = even_stages((229376 - kS - kOut) / kStage, 4);
    static constexpr int S0 = kStages * kStage, O0 = S0 + kS;
    static constexpr int W = O0 + kOut;        // 2 blocks of 8 rows x 128 bytes
    static constexpr int z0 = W + 2048;        // float[64 KB]
    static constexpr int bars = z0 + 512;
    static constexpr int total = bars + 512;
    static_assert(total >= W + 2 * 1024 + 1024, "the product's last read of W ends in the block's shared memory");
    static_assert(kStages >= 2 && total <= 232448, "query pass: shared memory");
};

template <int KB, int VB>
__global__ void __launch_bounds__(kQueryThreads, 1)
cross_query_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
               const __grid_constant__ CUtensorMap tm_dq, const char* __restrict__ image, float* rec, Rows rows, int Dk,
               int slots, int* err) {
    using SM = QuerySmem<KB, VB>;
    constexpr int NS = SM::kStages;
    constexpr uint32_t kY = 0, kR = 128 * KB, kW = kR + 64 * VB, kX = kW + 16;  // TMEM: two Y, R, r's 16, the halves' sums
    constexpr uint32_t kCols = kX + 8 <= 256 ? 256 : 512;
    extern __shared__ __align__(1024) uint8_t smem[];
    struct Bars {
        uint64_t full[4], empty[4], staged, out_free[2], s_full, s_empty, y_done[2], y_free[2], x_ready[4], w_ready[2], r_done[2], sums_done,
            r_flushed, final_mma, final_r;
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
            mbar_init(&bar->empty[s], 2);  // R's product and r's
            mbar_init(&bar->x_ready[s], 8);  // a stage's: a group may be a chunk ahead of R's products where the ring has four
        }
        mbar_init(&bar->staged, 8);
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bar->y_done[g], 1);
            mbar_init(&bar->y_free[g], 8);
            mbar_init(&bar->w_ready[g], 8);
            mbar_init(&bar->r_done[g], 1);
            mbar_init(&bar->out_free[g], 1);
        }
        mbar_init(&bar->s_full, 1);
        mbar_init(&bar->s_empty, 17);  // the products and the compute warps (z)
        mbar_init(&bar->sums_done, 2);  // a period's last products of R and of r
        mbar_init(&bar->r_flushed, 8);
        mbar_init(&bar->final_mma, 1);
        mbar_init(&bar->final_r, 1);
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

    if (warp < 4) reg_dec<56>();
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
                for (int b = 0; b < KB; ++b) tma_load_3d(st + b * T, &tm_q, 64 * b, w.row0(), w.bh, &bar->full[s]);
                for (int b = 0; b < VB; ++b) tma_load_3d(st + SM::kDo + b * T, &tm_do, 64 * b, w.row0(), w.bh, &bar->full[s]);
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
        constexpr uint32_t id_y = idesc_bf16_f32(128, 64 * KB, 0, 0), id_r = idesc_bf16_f32(128, 64 * VB, 1, 1);
        const uint32_t aS = smem_u32(smem + SM::S0), aSl = aS + (uint32_t)image_part(KB, VB), t0 = uniform(tmem);
        const int n = uniform(w.left);
        bool ok = true, y_first = true, first = true;
        int yi = 0, heads = 0, flushes = 0;
        Walk wy = w;
        Period period;
        auto issue_y = [&]() {  // Y of chunk yi: dO is all it needs, so it runs a chunk ahead
            const int g = yi & 1, s = yi % NS;
            if (y_first) ok = ok && warp_wait(&bar->s_full, heads++ & 1, err);
            ok = ok && warp_wait(&bar->full[s], (yi / NS) & 1, err) && warp_wait(&bar->y_free[g], ((yi >> 1) & 1) ^ 1, err);
            if (!ok) return;
            tc_fence_after();
            y_first = uniform(wy.last());
            if (elect_one()) {
                const uint32_t aD = smem_u32(smem + s * SM::kStage + SM::kDo), acc = t0 + kY + 64 * KB * g;
#pragma unroll
                for (int kk = 0; kk < 4 * VB; ++kk) {
                    mma_ss(acc, desc_k(aD, kk, T), desc_k(aS, kk, 8192 * KB), id_y, kk > 0);
                    mma_ss(acc, desc_k(aD, kk, T), desc_k(aSl, kk, 8192 * KB), id_y, 1);
                }
                mma_commit(&bar->y_done[g]);
                if (y_first) mma_commit(&bar->s_empty);
            }
            __syncwarp();
            wy.next();
            ++yi;
        };
        for (int i = 0; i < n && ok; ++i, w.next()) {
            const int s = i % NS;
            if (yi <= i) issue_y();
            ok = ok && warp_wait(&bar->x_ready[s], (i / NS) & 1, err);
            if (first && flushes > 0) ok = ok && warp_wait(&bar->r_flushed, (flushes - 1) & 1, err);
            if (!ok) break;
            tc_fence_after();
            const bool close = uniform(period.close(w));
            if (elect_one()) {
                const uint32_t st = smem_u32(smem + s * SM::kStage), aD = st + SM::kDo;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(t0 + kR, desc_mn(st, kk, T), desc_mn(aD, kk, T), id_r, !first || kk > 0);
                mma_commit(&bar->empty[s]);
                if (close) mma_commit(&bar->sums_done);
            }
            __syncwarp();
            first = close;
            if (first) ++flushes;
            // the next chunk's Y (its group's previous chunk, i - 1, is through), unless it needs the next head's S, for
            // which all of this head's chunks have to be through
            if (i + 1 < n && yi == i + 1 && !y_first) issue_y();
        }
        if (elect_one()) {
            mma_commit(&bar->final_mma);  // every product is complete before the accumulators are given back
            mbar_wait(&bar->final_mma, 0, err, LA_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == 3) {
        // r's products are ready later than R's, and their own thread's: behind one that waits for the other group's X they
        // held each group back until the other had caught up (358 us of B=2 H=16 N=32768 128 x 128)
        constexpr uint32_t id_w = idesc_bf16_f32(128, 16, 1, 0);
        const uint32_t aW = smem_u32(smem + SM::W), t0 = uniform(tmem);
        const int n = uniform(w.left);
        bool first = true;
        int flushes = 0;
        Period period;
        for (int i = 0; i < n; ++i, w.next()) {
            const int g = i & 1, s = i % NS;
            if (!warp_wait(&bar->w_ready[g], (i >> 1) & 1, err)) break;
            if (first && flushes > 0 && !warp_wait(&bar->r_flushed, (flushes - 1) & 1, err)) break;
            tc_fence_after();
            const bool close = uniform(period.close(w));
            if (elect_one()) {
                const uint32_t st = smem_u32(smem + s * SM::kStage);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) mma_ss(t0 + kW, desc_mn(st, kk, T), desc_k(aW, kk, 1024), id_w, !first || kk > 0);
                mma_commit(&bar->empty[s]);
                if (close) mma_commit(&bar->sums_done);
                mma_commit(&bar->r_done[g]);
            }
            __syncwarp();
            first = close;
            if (first) ++flushes;
        }
        if (elect_one()) {
            mma_commit(&bar->final_r);  // as above
            mbar_wait(&bar->final_r, 0, err, LA_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == 2) {
        if (lane == 0) {  // stores
            for (int i = 0; w.more(); w.next(), ++i) {
                if (!mbar_wait(&bar->staged, i & 1, err, LA_ERR_TIMEOUT)) break;
                check_copy(0, w.row0(), rows.M, w.bh, rows.heads());
                for (int b = 0; b < KB; ++b) tma_store_3d(&tm_dq, smem + SM::O0 + b * T, 64 * b, w.row0(), w.bh);
                bulk_commit();
                bulk_wait_read_all();
                mbar_arrive(&bar->out_free[i & 1]);
            }
            bulk_wait_all();
        }
    } else if (warp >= 4) {
        reg_inc<104>();
        constexpr int kHalf = 32 * KB;  // columns of this thread: its half of row r
        const int g = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, r = 32 * (warp & 3) + lane, pair = 1 + 4 * g + (warp & 3);
        const int c0 = kHalf * half, blk = (c0 >> 6) * T, lc0 = (c0 >> 3) & 7;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, acc = tmem + kY + 64 * KB * g + c0 + lanes;
        const uint32_t sums = tmem + kX + 4 * g + lanes;  // columns: den of either half, t of either half
        int i = 0, heads = 0, flushes = 0;
        bool first = true, ok = true, begun = false;  // begun: the record holds periods of this head
        Period period;
        for (; w.more(); w.next(), ++i) {
            // every head's, whether or not it has a chunk of this group
            if (first) ok = warp_wait(&bar->s_full, heads++ & 1, err);
            const bool last = first = w.last(), close = period.close(w);
            if ((i & 1) == g) {
                const int s = i % NS;
                uint8_t* st = smem + s * SM::kStage;
                ok = ok && warp_wait(&bar->full[s], (i / NS) & 1, err);
                // phi of the half row, its part of the normaliser
                float2 p[kHalf / 2], s2 = both(0.f);
#pragma unroll
                for (int c = 0; c < kHalf / 8; ++c) {
                    const uint4 x = *reinterpret_cast<const uint4*>(st + blk + swz(r, lc0 + c));
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                    float2 zv[4];
                    Pairs<float>::get(zs + c0 + 8 * c, reinterpret_cast<float2(&)[2]>(zv[0]));
                    Pairs<float>::get(zs + c0 + 8 * c + 4, reinterpret_cast<float2(&)[2]>(zv[2]));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[4 * c + e] = phi2(u[e]);
                        s2 = fma2(p[4 * c + e], zv[e], s2);
                    }
                }
                tmem_put(sums + half, s2.x + s2.y);
                if (!(ok = pair_all(pair, ok))) break;  // both halves are in
                const float inv = over(tmem_sum2(sums)), xi = r < w.rows() ? inv : 0.f;
                // X (rows behind the last query and padded columns, which hold phi(0): 0)
#pragma unroll
                for (int c = 0; c < kHalf / 8; ++c) {
                    uint4 h, l;
                    uint32_t *hw = reinterpret_cast<uint32_t*>(&h), *lw = reinterpret_cast<uint32_t*>(&l);
                    const float2 k = both(c0 + 8 * c < Dk ? xi : 0.f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (KB == 1)
                            split2(mul2(p[4 * c + e], k), hw[e], lw[e]);
                        else
                            hw[e] = pack2(mul2(p[4 * c + e], k));
                    }
                    *reinterpret_cast<uint4*>(st + blk + swz(r, lc0 + c)) = h;
                    if (KB == 1) *reinterpret_cast<uint4*>(st + SM::kLo + swz(r, lc0 + c)) = l;
                }
                fence_proxy_async_smem();
                warp_arrive(&bar->x_ready[s]);
                // t = phi(q) . Y / den
                ok = warp_wait(&bar->y_done[g], (i >> 1) & 1, err);
                tc_fence_after();
                s2 = both(0.f);
#pragma unroll
                for (int b = 0; b < 2 * KB; ++b) {
                    uint32_t y[16];
                    tmem_ld16(acc + 16 * b, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        s2 = fma2(p[8 * b + e], make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), s2);
                }
                tmem_put(sums + 2 + half, s2.x + s2.y);
                if (i > 0) ok = ok && warp_wait(&bar->r_done[(i - 1) & 1], ((i - 1) >> 1) & 1, err);  // W has been read
                if (!(ok = pair_all(pair, ok))) break;
                const float t = tmem_sum2(sums + 2) * inv;
                if (half == 0) {
                    uint32_t th, tl;
                    split2(make_float2(-t, 0.f), th, tl);
                    uint8_t* at = smem + SM::W + (r >> 6) * 1024 + (r & 7) * 2;
                    const int lc = (r & 63) >> 3;  // rows 0 and 1 of the operand
                    *reinterpret_cast<uint16_t*>(at + swz(0, lc)) = (uint16_t)th;
                    *reinterpret_cast<uint16_t*>(at + swz(1, lc)) = (uint16_t)tl;
                    fence_proxy_async_smem();
                }
                warp_arrive(&bar->w_ready[g]);
                // dq, packed until the tile of outputs is free
                const float2 mt = both(-t), iv = both(inv);  // t / den could overflow, inv phi' does not
                uint32_t dq[kHalf / 2];
#pragma unroll
                for (int b = 0; b < 2 * KB; ++b) {
                    uint32_t y[16];
                    tmem_ld16(acc + 16 * b, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        float2 zv[2];
                        Pairs<float>::get(zs + c0 + 16 * b + 2 * e, zv);
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            const int c = 2 * (e + o);
                            const float2 f = p[8 * b + e + o];
                            const float2 d = mul2(fma2(mt, zv[o], make_float2(__uint_as_float(y[c]), __uint_as_float(y[c + 1]))),
                                                  mul2(iv, make_float2(slope_of(f.x), slope_of(f.y))));
                            dq[8 * b + e + o] = pack2(d);
                        }
                    }
                }
                tc_fence_before();
                warp_arrive(&bar->y_free[g]);
                // the tile of outputs is free once the chunk before has been stored
                if (!(ok = pair_all(pair, i == 0 || warp_wait(&bar->out_free[(i - 1) & 1], ((i - 1) >> 1) & 1, err)))) break;
                const bool alive = any_key<KB>(zs);  // asked here: kept over the chunk it is a register too many (473 us to 487)
#pragma unroll
                for (int c = 0; c < kHalf / 8; ++c)
                    *reinterpret_cast<uint4*>(smem + SM::O0 + blk + swz(r, lc0 + c)) =
                        alive ? make_uint4(dq[4 * c], dq[4 * c + 1], dq[4 * c + 2], dq[4 * c + 3]) : make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                warp_arrive(&bar->staged);
                if (close) {  // the sums of this period
                    // The period before may be the other group's, whose additions to the record have to be in.  (Phases that this
                    // group has skipped are complete: those of earlier heads, as this head's S waited for every warp to be through
                    // with them; of this head, r_flushed's before the last, as R of the chunk before this one, whose products
                    // were issued before this chunk's Y, waited for it; sums_done's, as the last of r_flushed follows them.)
                    const bool in = !begun || warp_wait(&bar->r_flushed, (flushes - 1) & 1, err);
                    if (!(ok = pair_all(pair, in && warp_wait(&bar->sums_done, flushes & 1, err)))) break;
                    tc_fence_after();
                    if (LA_DCHECK((int)blockIdx.x + w.bh < slots)) {
                        float* out = rec + (size_t)(blockIdx.x + w.bh) * record_floats(VB);
                        tmem_row_to_record<32 * VB>(tmem + kR + 32 * VB * half + lanes, out + (size_t)r * 64 * VB + 32 * VB * half, begun);
                        uint32_t c[16];
                        tmem_ld16(tmem + kW + lanes, c);
                        tmem_ld_wait();
                        if (half == 0) {
                            float* to = out + 128 * 64 * VB + r;
                            *to = (begun ? *to : 0.f) + (__uint_as_float(c[0]) + __uint_as_float(c[1]));
                        }
                    }
                    tc_fence_before();
                    warp_arrive(&bar->r_flushed);
                }
            }
            if (close) ++flushes, begun = !last;
            if (last) {  // z is no longer read
                warp_arrive(&bar->s_empty);
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
// K and V have rings of their own, as they are free at different times: K (phi's bf16 copy in place) once its product is
// through, V, whose product starts as it lands, once dk (KB > VB: dv) has been stored from its place; the other output has a
// tile of its own.  With both outputs stored from one stage's tiles a stage waited 2,400 cycles for its stores and then
// 6,500 for its loads, of 14,000 in all (190 us of B=2 H=16 N=32768 128 x 128 instead of 183).  phi(K) enters dv's product
// rounded once: its errors are independent from column to column of R, whose entries are not.  phi'(k) is formed from k itself.
// Two groups of eight warps, half a row to a thread.
constexpr int kKeyThreads = 640;  // warp 0 TMA loads, 1 MMA, 2-17 two compute groups, 18 TMA stores, 19 zeros behind the lengths

template <int KB, int VB>
struct KeySmem {
    static constexpr int kK = KB * T, kV = VB * T, kOut = KB <= VB ? kV : kK, kR = 2 * (int)image_part(KB, VB);
    static constexpr int kStages = even_stages((229376 - kR - kOut) / (kK + kV), 4);
    static constexpr int V0 = kStages * kK, O0 = V0 + kStages * kV, R0 = O0 + kOut, r0 = R0 + kR, bars = r0 + 512, total = bars + 512;
    static_assert(kStages >= 2 && total <= 232448, "key pass: shared memory");
};

template <int KB, int VB>
__global__ void __launch_bounds__(kKeyThreads, 1)
cross_key_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
             const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv, const char* __restrict__ image,
             uint4* dk, uint4* dv, Rows keys, int Dk, int Dv, int* err) {
    using SM = KeySmem<KB, VB>;
    constexpr int NS = SM::kStages;
    constexpr uint32_t kSet = 64 * (KB + VB);  // TMEM of a group: dK without r and phi', then dV
    constexpr uint32_t kCols = 2 * kSet <= 256 ? 256 : 512;
    extern __shared__ __align__(1024) uint8_t smem[];
    struct Bars {
        uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], dk_staged[4], dv_staged[2], out_free[2], s_full, s_empty, ready[2], k_done[2], v_done[2],
            acc_free[2], final_mma;
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
            mbar_init(&bar->k_full[s], 1);
            mbar_init(&bar->k_empty[s], 1);
            mbar_init(&bar->v_full[s], 1);
            mbar_init(&bar->v_empty[s], 1);
            mbar_init(&bar->dk_staged[s], 8);  // a stage's: a group may be a chunk ahead of the stores where the ring has four
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bar->dv_staged[g], 8);
            mbar_init(&bar->ready[g], 8);
            mbar_init(&bar->k_done[g], 1);
            mbar_init(&bar->v_done[g], 1);
            mbar_init(&bar->acc_free[g], 8);
            mbar_init(&bar->out_free[g], 1);
        }
        mbar_init(&bar->s_full, 1);
        mbar_init(&bar->s_empty, 17);  // the products and the compute warps (r)
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
                check_copy(0, w.row0(), keys.M, w.bh, keys.heads());
                if (!mbar_wait(&bar->v_empty[s], ((i / NS) & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                mbar_arrive_expect_tx(&bar->v_full[s], VB * T);
                for (int b = 0; b < VB; ++b)
                    tma_load_3d(smem + SM::V0 + s * SM::kV + b * T, &tm_v, 64 * b, w.row0(), w.bh, &bar->v_full[s]);
                if (!mbar_wait(&bar->k_empty[s], ((i / NS) & 1) ^ 1, err, LA_ERR_TIMEOUT)) {
                    mbar_drain(bar->v_full, NS, i + 1, err, LA_ERR_TIMEOUT);
                    break;
                }
                mbar_arrive_expect_tx(&bar->k_full[s], KB * T);
                for (int b = 0; b < KB; ++b) tma_load_3d(smem + s * SM::kK + b * T, &tm_k, 64 * b, w.row0(), w.bh, &bar->k_full[s]);
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
            mbar_drain(bar->v_full, NS, i, err, LA_ERR_TIMEOUT);  // no copy is left in flight
            mbar_drain(bar->k_full, NS, i, err, LA_ERR_TIMEOUT);
            mbar_drain(&bar->s_full, 1, heads, err, LA_ERR_TIMEOUT);
        }
    } else if (warp == 1) {
        constexpr uint32_t id_k = idesc_bf16_f32(128, 64 * KB, 0, 0), id_v = idesc_bf16_f32(128, 64 * VB, 0, 1);
        const uint32_t aR = smem_u32(smem + SM::R0), aRl = aR + (uint32_t)image_part(KB, VB), t0 = uniform(tmem);
        const int n = uniform(w.left);
        int vi = 0, heads = 0;
        Walk wv = w;  // V R^T runs a chunk ahead
        bool v_first = true, ok = true;
        auto issue_k = [&]() {  // dK without r and phi' of chunk vi
            const int g = vi & 1, s = vi % NS;
            if (v_first) ok = ok && warp_wait(&bar->s_full, heads++ & 1, err);
            ok = ok && warp_wait(&bar->v_full[s], (vi / NS) & 1, err) && warp_wait(&bar->acc_free[g], ((vi >> 1) & 1) ^ 1, err);
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t aV = smem_u32(smem + SM::V0 + s * SM::kV), acc = t0 + kSet * g;
#pragma unroll
                for (int kk = 0; kk < 4 * VB; ++kk) {
                    mma_ss(acc, desc_k(aV, kk, T), desc_k(aR, kk, 8192 * KB), id_k, kk > 0);
                    mma_ss(acc, desc_k(aV, kk, T), desc_k(aRl, kk, 8192 * KB), id_k, 1);
                }
                mma_commit(&bar->k_done[g]);
            }
            __syncwarp();
            v_first = uniform(wv.last());
            wv.next();
            ++vi;
        };
        for (int i = 0; i < n && ok; ++i, w.next()) {
            const int g = i & 1, s = i % NS;
            if (vi <= i) issue_k();
            if (!ok || !warp_wait(&bar->ready[g], (i >> 1) & 1, err)) break;
            tc_fence_after();
            const bool last = uniform(w.last());
            if (elect_one()) {
                const uint32_t aK = smem_u32(smem + s * SM::kK), acc = t0 + kSet * g + 64 * KB;
#pragma unroll
                for (int kk = 0; kk < 4 * KB; ++kk) {
                    mma_ss(acc, desc_k(aK, kk, T), desc_mn(aR, kk, 8192 * KB), id_v, kk > 0);
                    mma_ss(acc, desc_k(aK, kk, T), desc_mn(aRl, kk, 8192 * KB), id_v, 1);
                }
                mma_commit(&bar->v_done[g]);
                mma_commit(&bar->k_empty[s]);
                if (last) mma_commit(&bar->s_empty);
            }
            __syncwarp();
            // the next chunk's, unless it needs the next head's R, for which this head has to be through
            if (i + 1 < n && vi == i + 1 && !v_first) issue_k();
        }
        if (elect_one()) {
            mma_commit(&bar->final_mma);  // every product is complete before the accumulators are given back
            mbar_wait(&bar->final_mma, 0, err, LA_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp < 18) {
        constexpr int kHalfK = 32 * KB, kHalfV = 32 * VB;  // columns of this thread: its half of row r
        const int g = (warp - 2) >> 3, half = ((warp - 2) >> 2) & 1, r = 32 * (warp & 3) + lane;
        const int ck = kHalfK * half, cv = kHalfV * half;
        const uint32_t acc = tmem + kSet * g + ((uint32_t)(32 * (warp & 3)) << 16);
        int i = 0, heads = 0;
        bool first = true;
        for (; w.more(); w.next(), ++i) {
            // every head's, whether or not it has a chunk of this group
            if (first && !warp_wait(&bar->s_full, heads++ & 1, err)) break;
            const bool last = first = w.last();
            if ((i & 1) == g) {
                const int s = i % NS;
                const bool live = r < w.rows();
                uint8_t *st = smem + s * SM::kK, *own = smem + SM::V0 + s * SM::kV, *out = smem + SM::O0;
                uint8_t *to_k = KB <= VB ? own : out, *to_v = KB <= VB ? out : own;
                if (!warp_wait(&bar->k_full[s], (i / NS) & 1, err)) break;
                uint4 k[kHalfK / 8];
#pragma unroll
                for (int c = 0; c < kHalfK / 8; ++c) {
                    uint4* at = reinterpret_cast<uint4*>(st + (ck >> 6) * T + swz(r, ((ck >> 3) & 7) + c));
                    uint4 x = k[c] = *at;
                    uint32_t* p = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = pack2(phi2(p[e]));
                    *at = x;
                }
                fence_proxy_async_smem();
                warp_arrive(&bar->ready[g]);
                if (!warp_wait(&bar->k_done[g], (i >> 1) & 1, err)) break;
                // the tile of outputs is free once the chunk before has been stored from it
                if (KB > VB && i > 0 && !warp_wait(&bar->out_free[(i - 1) & 1], ((i - 1) >> 1) & 1, err)) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < kHalfK / 32; ++b) {
                    uint32_t y[32];
                    tmem_ld32(acc + ck + 32 * b, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 x;
                        uint32_t* o = reinterpret_cast<uint32_t*>(&x);
                        const uint32_t* kw = reinterpret_cast<const uint32_t*>(&k[4 * b + c]);
                        float2 rr[4];
                        Pairs<float>::get(rs + ck + 32 * b + 8 * c, reinterpret_cast<float2(&)[2]>(rr[0]));
                        Pairs<float>::get(rs + ck + 32 * b + 8 * c + 4, reinterpret_cast<float2(&)[2]>(rr[2]));
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // formed again, and not as phi2 forms it: the compiler would keep phi2's exponentials, 64
                            // registers (184 us of B=2 H=16 N=32768 128 x 128 then, 168 so)
                            const float2 low = mul2(make_float2(min_nan(bf_lo(kw[e]), 0.f), min_nan(bf_hi(kw[e]), 0.f)),
                                                    both(1.4426950408889634f));
                            const float2 slope = make_float2(ex2_approx(low.x), ex2_approx(low.y));
                            const float2 d = mul2(norm::add2(make_float2(__uint_as_float(y[8 * c + 2 * e]), __uint_as_float(y[8 * c + 2 * e + 1])),
                                                             rr[e]), slope);
                            o[e] = pack2(d);
                        }
                        if (!live) x = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(to_k + ((ck + 32 * b) >> 6) * T + swz(r, (((ck + 32 * b) >> 3) & 7) + c)) = x;
                    }
                }
                fence_proxy_async_smem();
                warp_arrive(&bar->dk_staged[s]);
                if (!warp_wait(&bar->v_done[g], (i >> 1) & 1, err)) break;
                if (KB <= VB && i > 0 && !warp_wait(&bar->out_free[(i - 1) & 1], ((i - 1) >> 1) & 1, err)) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < kHalfV / 32; ++b) {
                    uint32_t y[32];
                    tmem_ld32(acc + 64 * KB + cv + 32 * b, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 x;
                        uint32_t* o = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = pack_bf16x2(__uint_as_float(y[8 * c + 2 * e]), __uint_as_float(y[8 * c + 2 * e + 1]));
                        if (!live) x = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(to_v + ((cv + 32 * b) >> 6) * T + swz(r, (((cv + 32 * b) >> 3) & 7) + c)) = x;
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                warp_arrive(&bar->acc_free[g]);
                warp_arrive(&bar->dv_staged[g]);
            }
            if (last) {  // r is no longer read
                warp_arrive(&bar->s_empty);
            }
        }
    } else if (warp == 19) {
        // the chunks behind the lengths (rows behind one inside a chunk are the compute warps'): this block's share of them
        if (keys.lens) {
            Span d = span_of(keys, kRowChunk, true, blockIdx.x, gridDim.x);
            for (; d.left > 0; --d.left) {
                const int b = d.bh / keys.Hk, row = ((keys.live(b) + kRowChunk - 1) / kRowChunk + d.i) * kRowChunk;
                const int n = min(kRowChunk, keys.M - row);
                const size_t at = (size_t)d.bh * keys.M + row;
                LA_DCHECK(d.bh < keys.heads() && n > 0);
                for (int x = lane; x < n * Dk / 8; x += 32) dk[at * Dk / 8 + x] = make_uint4(0u, 0u, 0u, 0u);
                for (int x = lane; x < n * Dv / 8; x += 32) dv[at * Dv / 8 + x] = make_uint4(0u, 0u, 0u, 0u);
                if (d.left == 1 || ++d.i < keys.chunks(b, kRowChunk, true)) continue;
                d.i = 0;
                do ++d.bh;  // ends: another chunk is left
                while (keys.chunks(d.bh / keys.Hk, kRowChunk, true) == 0);
            }
        }
    } else if (lane == 0) {
        for (int i = 0; w.more(); w.next(), ++i) {  // stores: a tile is free once its output has been read
            const int s = i % NS;
            const uint8_t *own = smem + SM::V0 + s * SM::kV, *out = smem + SM::O0;
            const uint8_t *of_k = KB <= VB ? own : out, *of_v = KB <= VB ? out : own;
            check_copy(0, w.row0(), keys.M, w.bh, keys.heads());
            if (!mbar_wait(&bar->dk_staged[s], (i / NS) & 1, err, LA_ERR_TIMEOUT)) break;
            for (int b = 0; b < KB; ++b) tma_store_3d(&tm_dk, of_k + b * T, 64 * b, w.row0(), w.bh);
            bulk_commit();
            if (!mbar_wait(&bar->dv_staged[i & 1], (i >> 1) & 1, err, LA_ERR_TIMEOUT)) break;
            for (int b = 0; b < VB; ++b) tma_store_3d(&tm_dv, of_v + b * T, 64 * b, w.row0(), w.bh);
            bulk_commit();
            bulk_wait_read_all_but_one();
            mbar_arrive(KB <= VB ? &bar->v_empty[s] : &bar->out_free[i & 1]);
            bulk_wait_read_all();
            mbar_arrive(KB <= VB ? &bar->out_free[i & 1] : &bar->v_empty[s]);
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
        CR_TRY(tc_join(kCentred, nullptr, a.S, a.z, ws + l.S, nullptr, nullptr, nullptr, keys, kSumRows, 1, s, st));
    } else {
        CR_TRY(tc_sums(a.k, a.v, keys, rec, l.sum_ctas, s, st));
        CR_TRY(tc_join(kCentred, rec, nullptr, nullptr, ws + l.S, nullptr, nullptr, nullptr, keys, kSumRows, l.sum_ctas, s, st));
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
        CR_TRY(tc_join(kGradSums, rec, nullptr, nullptr, ws + l.R, ws + l.S, nullptr, nullptr, rows, kRowChunk, l.query_ctas, s, st));
        return tc_run("cross_key_tc", key, dim3(l.key_ctas), kKeyThreads, ks, st, tk, tv, tdk, tdv, (const char*)ws + l.R, (uint4*)a.dk, (uint4*)a.dv,
                      keys, s.Dk, s.Dv, err);
    };
    cudaError_t e;
    switch (2 * blocks64(s.Dk) + blocks64(s.Dv)) {
        case 3: e = go(cross_query_tc<1, 1>, QuerySmem<1, 1>::total, cross_key_tc<1, 1>, KeySmem<1, 1>::total); break;
        case 4: e = go(cross_query_tc<1, 2>, QuerySmem<1, 2>::total, cross_key_tc<1, 2>, KeySmem<1, 2>::total); break;
        case 5: e = go(cross_query_tc<2, 1>, QuerySmem<2, 1>::total, cross_key_tc<2, 1>, KeySmem<2, 1>::total); break;
        default: e = go(cross_query_tc<2, 2>, QuerySmem<2, 2>::total, cross_key_tc<2, 2>, KeySmem<2, 2>::total); break;
    }
    return e;
}

}  // namespace cross
}  // namespace la
