// tc_cross.cu -- tensor-core kernels of cross attention forward: the sums over the keys, their join, the queries' answers.
//
//   cross_sums_tc   S = phi(K)^T V and z = phi(K)^T 1 of each block's share of the keys      records
//   cross_join_tc   a head's records added up in a fixed order                              image of (S, z)
//   cross_apply_tc  o = phi(Q) S / (phi(Q) z)                                                outputs
//
// All three are bound by memory: a chunk of 128 rows of 128-wide q and o (or k and v) is 64 KB, 1.45 us of an SM's share of
// the copy rate, against 0.35 us for its product.  What it takes to come near is loads in flight while the arithmetic of
// earlier chunks goes on, so tiles come through rings of TMA stages, and two groups of warps (eight each in the sums, four in
// the answers) work on alternate chunks, one waiting for its product while the other evaluates phi.  phi(k) enters the sums
// as two bf16 parts, so that S is good to 2^-17 of its terms: dq in the gradient is a small difference of products with S.  z adds
// the same parts, so that the two are sums of one phi.
// Measured, of the 6.79 TB/s a copy reaches: sums over 8 heads of 131,071 keys 105 us (0.75), answers to 2,097,152 queries
// of 16 heads 165 us (0.96), both 128 x 128.
#include <cudaTypedefs.h>

#include "tc_cross.cuh"

namespace la {
namespace cross {
namespace {

// ------------------------------------------------------------------ sums over the keys
// A stage holds a chunk of 64 rows: K (phi's hi part in place) and V.  phi's lo part: for KB = 1 in the stage, hi and lo being the
// two 64-row halves of one 128-row product; for KB = 2 in a ring of its own, held only while the products run.  An accumulator
// in tensor memory takes kPeriod chunks only: the products add with truncation, half a unit in the last place each and always the same way (131,072 keys summed in one
// accumulator to a block were 2e-5 off).  The compute warps then add it to sums of their own, in registers and rounded
// to nearest, while the other accumulator takes the next period: a warp has 32 rows and a quarter of the columns.
constexpr int kSumThreads = 576;  // warp 0 TMA, 1 MMA, 2-17 two compute groups of eight
constexpr int kPeriod = 4;
constexpr uint32_t kNone = 0xff80ff80u;  // -inf, -inf

template <int KB, int VB>
struct SumSmem {
    static constexpr int kTile = 8192;  // 64 rows of a block
    static constexpr int kV = 2 * kTile, kStage = kV + VB * kTile;  // K: two blocks, or phi's parts
    static constexpr int kLos = KB == 2 ? 3 : 0, kRoom = 212992 - kLos * 2 * kTile;
    static constexpr int kStages = even_stages(kRoom / kStage, 8);
    static constexpr int lo0 = kStages * kStage;
    static constexpr int zpart = lo0 + kLos * 2 * kTile;      // float[2][16][64 KB]
    static constexpr int bars = zpart + 2 * 16 * 64 * KB * 4;
    static constexpr int total = bars + 512;
};

template <int KB, int VB>
__global__ void __launch_bounds__(kSumThreads, 1)
cross_sums_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, float* __restrict__ rec, Rows keys,
              int Dk, int slots, int* err) {
    using SM = SumSmem<KB, VB>;
    constexpr int NS = SM::kStages, T = SM::kTile, kLos = KB == 2 ? SM::kLos : 1;
    extern __shared__ __align__(1024) uint8_t smem[];
    struct Bars {
        uint64_t full[8], ready[8], empty[8], lo_free[3], acc_done[2], flushed[2], z_ready[2], z_free[2], final_mma;
        uint32_t tmem;
        Span span;
    };
    static_assert(sizeof(Bars) <= 512, "barriers");
    Bars* bar = reinterpret_cast<Bars*>(smem + SM::bars);
    LA_DCHECK((smem_u32(smem) & 1023) == 0);
    float* zpart = reinterpret_cast<float*>(smem + SM::zpart);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 32) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->ready[s], 8);
            mbar_init(&bar->empty[s], 1);
        }
        for (int l = 0; l < SM::kLos; ++l) mbar_init(&bar->lo_free[l], 1);
        for (int a = 0; a < 2; ++a) {
            mbar_init(&bar->acc_done[a], 1);
            mbar_init(&bar->flushed[a], 16);
            mbar_init(&bar->z_ready[a], 16);
            mbar_init(&bar->z_free[a], 4);
        }
        mbar_init(&bar->final_mma, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(&bar->tmem, 128 * VB);
        tmem_relinquish();
    }
    pdl_enter();  // launched with programmatic dependent launch
    if (warp == 0) {
        const Span sp = span_of(keys, kSumRows, false, blockIdx.x, gridDim.x);
        if (lane == 0) bar->span = sp;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;
    Walk w(keys, kSumRows, bar->span);

    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            for (; w.more(); w.next(), ++i) {
                const int s = i % NS;
                if (!mbar_wait(&bar->empty[s], ((i / NS) & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                uint8_t* st = smem + s * SM::kStage;
                mbar_arrive_expect_tx(&bar->full[s], (KB + VB) * T);
                check_copy(0, w.row0(), keys.M, w.bh, keys.heads());
                for (int b = 0; b < KB; ++b) tma_load_3d(st + b * T, &tm_k, 64 * b, w.row0(), w.bh, &bar->full[s]);
                for (int b = 0; b < VB; ++b) tma_load_3d(st + SM::kV + b * T, &tm_v, 64 * b, w.row0(), w.bh, &bar->full[s]);
            }
            mbar_drain(bar->full, NS, i, err, LA_ERR_TIMEOUT);  // no copy is left in flight
        }
    } else if (warp == 1) {
        constexpr uint32_t id = idesc_bf16_f32(128, 64 * VB, 1, 1);
        const uint32_t lo = smem_u32(smem + SM::lo0), t0 = uniform(tmem);
        const int n = uniform(w.left);
        int period = 0, in = 0;  // chunks of the period so far
        for (int i = 0; i < n; ++i, w.next()) {
            const int s = i % NS, a = period & 1;
            if (!warp_wait(&bar->ready[s], (i / NS) & 1, err)) break;
            if (in == 0 && !warp_wait(&bar->flushed[a], ((period >> 1) & 1) ^ 1, err)) break;
            tc_fence_after();
            const bool close = uniform(in + 1 == kPeriod || w.last());
            if (elect_one()) {
                const uint32_t st = smem_u32(smem + s * SM::kStage), acc = t0 + 64 * VB * a;
#pragma unroll
                for (int kk = 0; kk < kSumRows / 16; ++kk) {
                    mma_ss(acc, desc_mn(st, kk, T), desc_mn(st + SM::kV, kk, T), id, in > 0 || kk > 0);
                    if (KB == 2) mma_ss(acc, desc_mn(lo + i % kLos * 2 * T, kk, T), desc_mn(st + SM::kV, kk, T), id, 1);
                }
                if (KB == 2) mma_commit(&bar->lo_free[i % kLos]);  // before empty: see the wait for it
                mma_commit(&bar->empty[s]);
                if (close) mma_commit(&bar->acc_done[a]);
            }
            __syncwarp();
            ++in;
            if (close) in = 0, ++period;
        }
        if (elect_one()) {
            mma_commit(&bar->final_mma);  // every product is complete before the accumulators are given back
            mbar_wait(&bar->final_mma, 0, err, LA_ERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        const int cw = warp - 2, group = cw >> 3, ct = (tid - 64) & 255;
        const int lc = (ct & 7) ^ ((ct >> 3) & 7), at = (ct >> 3) * 128 + (ct & 7) * 16;  // rows (ct >> 3) + 32 j
        constexpr int kOwn = 16 * VB;  // columns of this warp's sums, of the rows 32 (warp % 4) ..
        const int col0 = kOwn * (cw >> 2);
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        float2 zp[KB][4];
        float sum[kOwn];
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) zp[b][e] = norm::both(0.f);
#pragma unroll
        for (int e = 0; e < kOwn; ++e) sum[e] = 0.f;
        int i = 0, period = 0, flushed = 0, heads = 0;
        int in = 0;
        bool ok = true;
        auto flush = [&]() {  // the oldest period not yet added
            const int a = flushed & 1;
            ok = ok && warp_wait(&bar->acc_done[a], (flushed >> 1) & 1, err);
            if (!ok) return;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kOwn / 16; ++c) {
                uint32_t x[16];
                tmem_ld16(tmem + 64 * VB * a + col0 + 16 * c + lanes, x);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[16 * c + e] += __uint_as_float(x[e]);
            }
            tc_fence_before();
            warp_arrive(&bar->flushed[a]);
            ++flushed;
        };
        for (; w.more() && ok; w.next(), ++i) {
            if ((i & 1) == group) {
                const int s = i % NS, n = w.rows();
                if (!(ok = warp_wait(&bar->full[s], (i / NS) & 1, err))) break;
                // (this group has skipped the slot's phase before; it is complete, as full is, which waited for chunk i - NS or later)
                static_assert(NS <= 2 * kLos || KB == 1, "the slot's release before the last is older than this stage's");
                if (KB == 2 && !(ok = warp_wait(&bar->lo_free[i % kLos], ((i / kLos) & 1) ^ 1, err))) break;
                uint8_t* st = smem + s * SM::kStage + at;
                uint8_t* lo = KB == 2 ? smem + SM::lo0 + i % kLos * 2 * T + at : st + T;
                uint4 x[KB][2];
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[b][j] = *reinterpret_cast<const uint4*>(st + b * T + 4096 * j);
                if (n < kSumRows || (Dk & 63) != 0) {  // phi(-inf) is 0; masked here, the loop below has no branch
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (64 * b + 8 * lc >= Dk || (ct >> 3) + 32 * j >= n)
                                x[b][j] = make_uint4(kNone, kNone, kNone, kNone);
                }
#pragma unroll
                for (int b = 0; b < KB; ++b) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t* u = reinterpret_cast<uint32_t*>(&x[b][j]);
                        uint4 l;
                        uint32_t* ul = reinterpret_cast<uint32_t*>(&l);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            split2(phi2(u[e]), u[e], ul[e]);
                            zp[b][e] = norm::add2(zp[b][e], norm::add2(unpack2(u[e]), unpack2(ul[e])));
                        }
                        *reinterpret_cast<uint4*>(st + b * T + 4096 * j) = x[b][j];
                        *reinterpret_cast<uint4*>(lo + b * T + 4096 * j) = l;
                    }
                }
                if (n < kSumRows) {  // what lies behind the length may be anything
#pragma unroll
                    for (int b = 0; b < VB; ++b)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if ((ct >> 3) + 32 * j >= n)
                                *reinterpret_cast<uint4*>(st + SM::kV + b * T + 4096 * j) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                warp_arrive(&bar->ready[s]);
            }
            const bool last = w.last();
            if (++in < kPeriod && !last) continue;
            in = 0;
            ++period;
            while (ok && flushed < (last ? period : period - 1)) flush();
            if (!last || !ok) continue;
            // the head's record: this warp's sums, and z over the four lanes that share columns, then over the warps
            const int a = heads & 1, r = 32 * (warp & 3) + lane;
            if (!(ok = warp_wait(&bar->z_free[a], ((heads >> 1) & 1) ^ 1, err))) break;
            float* to = zpart + (a * 16 + cw) * 64 * KB + 8 * lc;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float z = e & 1 ? zp[b][e >> 1].y : zp[b][e >> 1].x;
                    z += __shfl_xor_sync(0xffffffffu, z, 9);
                    z += __shfl_xor_sync(0xffffffffu, z, 18);
                    if (lane < 8) to[64 * b + e] = z;
                    if (e & 1) zp[b][e >> 1] = norm::both(0.f);
                }
            warp_arrive(&bar->z_ready[a]);
            const bool slot = LA_DCHECK((int)blockIdx.x + w.bh < slots);
            float* out = rec + (size_t)(blockIdx.x + w.bh) * record_floats(VB);
#pragma unroll
            for (int e = 0; e < kOwn; e += 4) {
                if (slot) *reinterpret_cast<float4*>(out + (size_t)r * 64 * VB + col0 + e) = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
                sum[e] = sum[e + 1] = sum[e + 2] = sum[e + 3] = 0.f;
            }
            if (cw < 4) {
                if (!(ok = warp_wait(&bar->z_ready[a], (heads >> 1) & 1, err))) break;
                const int c = 32 * cw + lane;
                float z = 0.f;
                if (c < 64 * KB)
#pragma unroll
                    for (int x = 0; x < 16; ++x) z += zpart[(a * 16 + x) * 64 * KB + c];
                if (slot) out[128 * 64 * VB + c] = z;
                warp_arrive(&bar->z_free[a]);
            }
            ++heads;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 128 * VB);
    }
}

// ------------------------------------------------------------------ join
// A head's records (or a caller's state) to its image.  kLanes threads share a 16-byte chunk of the image, each taking every
// kLanes-th record; their sums are added in a fixed order.  The thread of a row's first chunk adds up the row's z, or r.
//
// Centred images are the gradient's.  dq = (Y - t z) / den and dk = R v + r are small where the values are alike, and what cancels
// there, the part of v that all keys have in common, would leave the rounding of S to 16 bits behind.  For any vector c
//   S' = S - z c^T,  Y' = S' dO,  t' = phi(q) . Y' / den = t - c . dO,  dq = (Y' - t' z) / den phi'(q),
//   r' = -sum x t',  r = r' - R c,
// so with c a weighted mean of the head's values, c = S[d,:] / z[d] for one row d, the common part is gone before anything is rounded
// to bf16.  c is kept in the image for the join of (R, r), which subtracts R c with R as the products have it.  It only has to be
// the same wherever it is used; one that is not finite counts as 0.  d is a row of no extreme z, the second largest of four: the
// largest may be a single key's, the smallest a few keys'.  (With S itself one key left 10 times the residue that fp32 leaves,
// and values of 250 times their spread a dq 1.5e-2 off; with the mean of the first record alone, 131,072 values that grow along the
// keys a dq 5.9e-3 off instead of 1.7e-3.)
template <int KB, int VB>
__device__ __forceinline__ float record_z(const float* p, int d) {
    p += 128 * 64 * VB + d;
    return KB == 1 ? p[0] + p[64] : p[0];
}

template <int KB, int VB, int kLanes, int kMode>
__global__ void __launch_bounds__(256)
cross_join_tc(const float* __restrict__ rec, const float* __restrict__ S, const float* __restrict__ z, char* __restrict__ image,
              const char* __restrict__ centre, float* __restrict__ S_out, float* __restrict__ z_out, Rows rows, int chunk, int ctas,
              int Dk, int Dv) {
    constexpr int kRow = 8 * VB, kOwn = 256 / kLanes;  // 16-byte chunks of a row; of a block
    constexpr bool kC = kMode == kCentred;
    constexpr int kParts = kC ? 19 : 9;  // v, z, and c, its z; odd
    __shared__ float part[kLanes > 1 ? kLanes : 1][kLanes > 1 ? kOwn : 1][kParts];
    pdl_enter();  // launched with programmatic dependent launch
    const int bh = blockIdx.x, x = threadIdx.x % kOwn, lane = threadIdx.x / kOwn;
    Range g{0, 0};
    if (rec) g = records_of(rows, chunk, bh, ctas);
    char* im = image + (size_t)bh * image_bytes(KB, VB);
    // row d, columns c8 .. c8 + 7
    const int at = blockIdx.y * kOwn + x, d = at / kRow, c8 = at % kRow * 8;
    float v[8], c[8], zs = 0.f, zc = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c[e] = 0.f;
    auto add = [&](const float* p, float (&to)[8]) {
        const float4 f = *reinterpret_cast<const float4*>(p), h = *reinterpret_cast<const float4*>(p + 4);
        to[0] += f.x, to[1] += f.y, to[2] += f.z, to[3] += f.w, to[4] += h.x, to[5] += h.y, to[6] += h.z, to[7] += h.w;
    };
    auto add_row = [&](const float* p, int row, float (&to)[8]) {  // of a record
        p += (size_t)row * 64 * VB + c8;
        add(p, to);
        if (KB == 1) add(p + 64 * 64 * VB, to);  // the sums of the lo parts
    };
    int dc = 0;  // the row of c: of four, by the first record's z, the second largest
    if (kC && (!rec || g.first <= g.last)) {
        const float* zf = rec ? rec + (size_t)(g.first + bh) * record_floats(VB) : z + (size_t)bh * Dk;
        float most = -1.f, next = -1.f;
        int top = 0;
#pragma unroll
        for (int i = 1; i < 8; i += 2) {
            const int r = Dk / 8 * i;
            const float f = rec ? record_z<KB, VB>(zf, r) : zf[r];
            if (f > most)
                next = most, dc = top, most = f, top = r;
            else if (f > next)
                next = f, dc = r;
        }
    }
    const bool with_z = kC || c8 == 0;
    if (!rec) {
        const float* Sh = S + (size_t)bh * Dk * Dv + c8;
        if (d < Dk) {
            if (c8 < Dv) add(Sh + (size_t)d * Dv, v);
            if (with_z) zs = z[(size_t)bh * Dk + d];
        }
        if (kC) {
            if (c8 < Dv) add(Sh + (size_t)dc * Dv, c);
            zc = z[(size_t)bh * Dk + dc];
        }
    } else {
#pragma unroll 4
        for (int i = g.first + lane; i <= g.last; i += kLanes) {
            const float* p = rec + (size_t)(i + bh) * record_floats(VB);
            add_row(p, d, v);
            if (with_z) zs += record_z<KB, VB>(p, d);
            if (kC) {
                add_row(p, dc, c);
                zc += record_z<KB, VB>(p, dc);
            }
        }
    }
    if constexpr (kLanes > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            part[lane][x][e] = v[e];
            if (kC) part[lane][x][9 + e] = c[e];
        }
        part[lane][x][8] = zs;
        if (kC) part[lane][x][17] = zc;
        __syncthreads();
        if (lane != 0) return;
        auto total = [&](int e) {
            float s = 0.f;
#pragma unroll
            for (int l = 0; l < kLanes; ++l) s += part[l][x][e];
            return s;
        };
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = total(e);
            if (kC) c[e] = total(9 + e);
        }
        zs = total(8);
        if (kC) zc = total(17);
    }
    if (S_out && d < Dk && c8 < Dv) {
        float* to = S_out + ((size_t)bh * Dk + d) * Dv + c8;
        *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
    if constexpr (kC) {
        const bool use = zc >= FLT_MIN && zc <= FLT_MAX;  // else no key, or one of infinity
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            c[e] /= zc;
            if (!use || !(fabsf(c[e]) <= FLT_MAX)) c[e] = 0.f;
            v[e] = fmaf(-zs, c[e], v[e]);
        }
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(make_float2(v[2 * e], v[2 * e + 1]), hi[e], lo[e]);
    const int off = (c8 >> 6) * (64 * KB * 128) + swz(d, c8 >> 3);
    *reinterpret_cast<uint4*>(im + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(im + image_part(KB, VB) + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if constexpr (kMode == kGradSums) {  // r = r' - R c
        const float* cs = image_centre(centre + (size_t)bh * image_bytes(KB, VB), KB, VB) + c8;
        float2 dot = norm::both(0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            dot = norm::fma2(norm::add2(unpack2(hi[e]), unpack2(lo[e])), *reinterpret_cast<const float2*>(cs + 2 * e), dot);
        float s = dot.x + dot.y;
#pragma unroll
        for (int o = kRow / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        zs -= s;
    }
    if (c8 == 0) {
        reinterpret_cast<float*>(im + 2 * image_part(KB, VB))[d] = zs;
        if (z_out && d < Dk) z_out[(size_t)bh * Dk + d] = zs;
    }
    if (kC && d == 0) {
        float* to = image_centre(im, KB, VB) + c8;
        *reinterpret_cast<float4*>(to) = make_float4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(c[4], c[5], c[6], c[7]);
    }
}

// ------------------------------------------------------------------ the queries' answers
// A stage holds a chunk of 128 queries: phi(Q) in place for the product, then the outputs for their store.  A thread owns
// a row.  S (its hi part) and z of the next head are copied while this head's chunks are worked on.  One part of phi(q) and of S
// is enough for an S that was summed from keys: its rows are alike, so that their roundings and phi's average out over the
// columns of a head (o is as far off as its own rounding, 1.6 times that where one key outweighs the others).  A caller's state may be any: kExact forms
// phi_hi S_hi + phi_hi S_lo + phi_lo S_hi (independent entries: 1.8 times as far off without).
constexpr int kApplyThreads = 352;  // warp 0 TMA loads, 1 MMA, 2-9 two compute groups, 10 TMA stores

template <int KB, int VB, bool kExact>
struct ApplySmem {
    static constexpr int kTile = 16384;  // 128 rows of a block
    static constexpr int kBufs = kExact ? 1 : 2;  // of S
    static constexpr int kS = (kExact ? 2 : 1) * (int)image_part(KB, VB);
    static constexpr int kLo = (KB > VB ? KB : VB) * kTile, kStage = kLo + (kExact ? KB * kTile : 0);
    static constexpr int kStages = even_stages((229376 - kBufs * kS) / kStage, 6);
    static constexpr int S0 = kStages * kStage;
    static constexpr int z0 = S0 + kBufs * kS;      // float[kBufs][64 KB]
    static constexpr int bars = z0 + kBufs * 256 * KB;
    static constexpr int total = bars + 512;
    static_assert(kStages >= 2 && total <= 232448, "apply: shared memory");
};

template <int KB, int VB, bool kExact>
__global__ void __launch_bounds__(kApplyThreads, 1)
cross_apply_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o, const char* __restrict__ image,
               Rows rows, int* err) {
    using SM = ApplySmem<KB, VB, kExact>;
    constexpr int NS = SM::kStages, T = SM::kTile, NB = SM::kBufs;
    extern __shared__ __align__(1024) uint8_t smem[];
    struct Bars {
        uint64_t full[6], empty[6], staged[6], s_full[2], s_empty[2], ready[2], done[2], final_mma;
        uint32_t tmem;
        Span span;
    };
    static_assert(sizeof(Bars) <= 512, "barriers");
    Bars* bar = reinterpret_cast<Bars*>(smem + SM::bars);
    LA_DCHECK((smem_u32(smem) & 1023) == 0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 32) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 1);
            mbar_init(&bar->staged[s], 4);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bar->s_full[g], 1);
            mbar_init(&bar->s_empty[g], 9);  // the products and the compute warps
            mbar_init(&bar->ready[g], 4);
            mbar_init(&bar->done[g], 1);
        }
        mbar_init(&bar->final_mma, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_o);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(&bar->tmem, 128 * VB);
        tmem_relinquish();
    }
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

    if (warp == 0) {
        if (lane == 0) {
            int i = 0, heads = 0;
            bool first = true;
            for (; w.more(); w.next(), ++i) {
                if (first) {
                    const int h = heads % NB;
                    if (!mbar_wait(&bar->s_empty[h], ((heads / NB) & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                    const char* im = image + (size_t)w.bh * image_bytes(KB, VB);
                    mbar_arrive_expect_tx(&bar->s_full[h], SM::kS + 256 * KB);
                    bulk_load(smem + SM::S0 + h * SM::kS, im, SM::kS, &bar->s_full[h]);
                    bulk_load(smem + SM::z0 + h * 256 * KB, im + 2 * image_part(KB, VB), 256 * KB, &bar->s_full[h]);
                    ++heads;
                }
                first = w.last();
                const int s = i % NS;
                if (!mbar_wait(&bar->empty[s], ((i / NS) & 1) ^ 1, err, LA_ERR_TIMEOUT)) break;
                mbar_arrive_expect_tx(&bar->full[s], KB * T);
                check_copy(0, w.row0(), rows.M, w.bh, rows.heads());
                for (int b = 0; b < KB; ++b) tma_load_3d(smem + s * SM::kStage + b * T, &tm_q, 64 * b, w.row0(), w.bh, &bar->full[s]);
            }
            mbar_drain(bar->full, NS, i, err, LA_ERR_TIMEOUT);  // no copy is left in flight
            mbar_drain(bar->s_full, NB, heads, err, LA_ERR_TIMEOUT);
        }
    } else if (warp == 1) {
        constexpr uint32_t id = idesc_bf16_f32(128, 64 * VB, 0, 1);
        const uint32_t t0 = uniform(tmem);
        const int n = uniform(w.left);
        int heads = 0;
        bool first = true;
        for (int i = 0; i < n; ++i, w.next()) {
            const int g = i & 1, s = i % NS;
            if (first) ++heads;
            const int h = (heads - 1) % NB;
            if (first && !warp_wait(&bar->s_full[h], ((heads - 1) / NB) & 1, err)) break;
            // phi(Q) is in place, and the group has read the outputs of its previous chunk
            if (!warp_wait(&bar->ready[g], (i >> 1) & 1, err)) break;
            tc_fence_after();
            first = uniform(w.last());
            if (elect_one()) {
                const uint32_t aQ = smem_u32(smem + s * SM::kStage), aS = smem_u32(smem + SM::S0 + h * SM::kS);
#pragma unroll
                for (int kk = 0; kk < 4 * KB; ++kk) {
                    mma_ss(t0 + 64 * VB * g, desc_k(aQ, kk, T), desc_mn(aS, kk, 8192 * KB), id, kk > 0);
                    if (kExact) {
                        mma_ss(t0 + 64 * VB * g, desc_k(aQ, kk, T), desc_mn(aS + (uint32_t)image_part(KB, VB), kk, 8192 * KB), id, 1);
                        mma_ss(t0 + 64 * VB * g, desc_k(aQ + SM::kLo, kk, T), desc_mn(aS, kk, 8192 * KB), id, 1);
                    }
                }
                mma_commit(&bar->done[g]);
                if (first) mma_commit(&bar->s_empty[h]);
            }
            __syncwarp();
        }
        if (elect_one()) {
            mma_commit(&bar->final_mma);  // every product is complete before the accumulators are given back
            mbar_wait(&bar->final_mma, 0, err, LA_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp < 10) {
        const int g = (warp - 2) >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t acc = tmem + 64 * VB * g + ((uint32_t)(32 * (warp & 3)) << 16);
        int i = 0, heads = 0;
        bool first = true, alive = true;
        for (; w.more(); w.next(), ++i) {
            const int h = (first ? heads : heads - 1) % NB;
            const float* zs = reinterpret_cast<const float*>(smem + SM::z0 + h * 256 * KB);
            // every head's, whether or not it has a chunk of this group: a wait that skips a phase can be let through by the one
            // before, and one that the next phase overtakes does not end, so each warp also says when it is through with a head
            if (first) {
                if (!warp_wait(&bar->s_full[h], (heads++ / NB) & 1, err)) break;
                alive = any_key<KB>(zs);
            }
            first = w.last();
            if ((i & 1) != g) {
                if (first) warp_arrive(&bar->s_empty[h]);
                continue;
            }
            const int s = i % NS;
            uint8_t* st = smem + s * SM::kStage;
            if (!warp_wait(&bar->full[s], (i / NS) & 1, err)) break;
            float2 den = norm::both(0.f);
#pragma unroll
            for (int b = 0; b < KB; ++b) {
#pragma unroll
                for (int lc = 0; lc < 8; ++lc) {
                    uint4* p = reinterpret_cast<uint4*>(st + b * T + swz(r, lc));
                    uint4 x = *p;
                    uint32_t *u = reinterpret_cast<uint32_t*>(&x), l[4];
                    float2 zv[4];
                    norm::Pairs<float>::get(zs + 64 * b + 8 * lc, reinterpret_cast<float2(&)[2]>(zv[0]));
                    norm::Pairs<float>::get(zs + 64 * b + 8 * lc + 4, reinterpret_cast<float2(&)[2]>(zv[2]));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = phi2(u[e]);
                        if (kExact) {
                            split2(f, u[e], l[e]);
                            den = norm::fma2(f, zv[e], den);
                        } else {
                            u[e] = pack2(f);
                            den = norm::fma2(unpack2(u[e]), zv[e], den);  // of the rounded phi, as the product has it
                        }
                    }
                    *p = x;
                    if (kExact) *reinterpret_cast<uint4*>(st + SM::kLo + b * T + swz(r, lc)) = make_uint4(l[0], l[1], l[2], l[3]);
                }
            }
            const float2 inv = norm::both(over(den.x + den.y));
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&bar->ready[g]);
            if (first) warp_arrive(&bar->s_empty[h]);  // z has been read
            if (!warp_wait(&bar->done[g], (i >> 1) & 1, err)) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2 * VB; ++b) {
                uint32_t o[32];
                tmem_ld32(acc + 32 * b, o);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint4 x;
                    uint32_t* u = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        u[e] = pack2(norm::mul2(make_float2(__uint_as_float(o[8 * c + 2 * e]), __uint_as_float(o[8 * c + 2 * e + 1])), inv));
                    if (!alive) x = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(st + (b >> 1) * T + swz(r, 4 * (b & 1) + c)) = x;
                }
            }
            fence_proxy_async_smem();
            warp_arrive(&bar->staged[s]);
        }
    } else if (lane == 0) {
        // stores: a stage is empty once its outputs have been read
        for (int i = 0; w.more(); w.next(), ++i) {
            const int s = i % NS;
            if (!mbar_wait(&bar->staged[s], (i / NS) & 1, err, LA_ERR_TIMEOUT)) break;
            check_copy(0, w.row0(), rows.M, w.bh, rows.heads());
            for (int b = 0; b < VB; ++b) tma_store_3d(&tm_o, smem + s * SM::kStage + b * T, 64 * b, w.row0(), w.bh);
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
        tmem_dealloc(tmem, 128 * VB);
    }
}

int ctas_for(long long heads, long long rows, int chunk) {  // a block to an SM, or to a chunk
    const long long chunks = heads * ((rows + chunk - 1) / chunk);
    return (int)(chunks < kSms ? chunks : kSms);
}

cudaError_t answers(const void* q, void* o, const char* image, bool exact, const la_cross_shape& s, cudaStream_t st) {
    const Rows rows = grouped_queries(s);
    CUtensorMap tq, to;
    if (!make_tmap_bf16_rows(&tq, q, rows.heads(), rows.M, s.Dk, kRowChunk) ||
        !make_tmap_bf16_rows(&to, o, rows.heads(), rows.M, s.Dv, kRowChunk))
        return cudaErrorInvalidValue;
    const int ctas = ctas_for(rows.heads(), rows.M, kRowChunk);
    auto go = [&](auto kern, size_t smem) {
        return tc_run("cross_apply_tc", kern, dim3(ctas), kApplyThreads, smem, st, tq, to, image, rows, device_error_word());
    };
#define LA_GO(KB, VB) \
    exact ? go(cross_apply_tc<KB, VB, true>, ApplySmem<KB, VB, true>::total) : go(cross_apply_tc<KB, VB, false>, ApplySmem<KB, VB, false>::total)
    switch (2 * blocks64(s.Dk) + blocks64(s.Dv)) {
        case 3: return LA_GO(1, 1);
        case 4: return LA_GO(1, 2);
        case 5: return LA_GO(2, 1);
        default: return LA_GO(2, 2);
    }
#undef LA_GO
}

}  // namespace

bool tc_ok(const la_cross_shape& s) { return s.dtype == LA_BF16; }

TcLayout tc_layout(const la_cross_shape& s, int op) {
    const int KB = blocks64(s.Dk), VB = blocks64(s.Dv);
    const size_t heads = (size_t)s.B * s.Hk, image = up(heads * image_bytes(KB, VB)), rec = record_floats(VB) * 4;
    TcLayout l{};
    if (op != LA_OP_CROSS_APPLY) {
        l.sum_ctas = ctas_for(heads, s.M, kSumRows);
        l.key_ctas = ctas_for(heads, s.M, kRowChunk);
        size_t most = l.sum_ctas;
        if (op == LA_OP_CROSS_BWD) {
            l.query_ctas = ctas_for(heads, query_rows(s), kRowChunk);
            if ((size_t)l.query_ctas > most) most = l.query_ctas;
        }
        l.bytes = up((most + heads) * rec);
    }
    l.S = l.bytes;
    l.bytes += image;
    if (op == LA_OP_CROSS_BWD) {
        l.R = l.bytes;
        l.bytes += image;
    }
    return l;
}
size_t tc_bytes(const la_cross_shape& s, int op) { return tc_layout(s, op).bytes; }

cudaError_t tc_sums(const void* k, const void* v, const Rows& keys, float* rec, int ctas, const la_cross_shape& s, cudaStream_t st) {
    CUtensorMap tk, tv;
    if (!make_tmap_bf16_rows(&tk, k, keys.heads(), keys.M, s.Dk, kSumRows) ||
        !make_tmap_bf16_rows(&tv, v, keys.heads(), keys.M, s.Dv, kSumRows))
        return cudaErrorInvalidValue;
    auto go = [&](auto kern, size_t smem) {
        return tc_run("cross_sums_tc", kern, dim3(ctas), kSumThreads, smem, st, tk, tv, rec, keys, s.Dk, ctas + keys.heads(),
                      device_error_word());
    };
    switch (2 * blocks64(s.Dk) + blocks64(s.Dv)) {
        case 3: return go(cross_sums_tc<1, 1>, SumSmem<1, 1>::total);
        case 4: return go(cross_sums_tc<1, 2>, SumSmem<1, 2>::total);
        case 5: return go(cross_sums_tc<2, 1>, SumSmem<2, 1>::total);
        default: return go(cross_sums_tc<2, 2>, SumSmem<2, 2>::total);
    }
}

cudaError_t tc_join(JoinMode mode, const float* rec, const float* S, const float* z, char* image, const char* centre, float* S_out,
                    float* z_out, const Rows& rows, int chunk, int ctas, const la_cross_shape& s, cudaStream_t st) {
    const int KB = blocks64(s.Dk), VB = blocks64(s.Dv);
    // few records to a head: a thread to a chunk; many (few heads): eight, with an eighth of the records each.  Gradients of N = M =
    // 262144 / heads with one and with eight, us: 64 x 64, 8 heads 132 and 91, 32 105 and 93, 76 89 and 91, 152 89 and 98; 128 x 128, 8
    // heads 167 and 144, 32 161 and 162, 38 147 and 153, 152 148 and 194.
    const bool many = rec && ctas > 4 * rows.heads();
    auto go = [&](auto kern, int own) {
        launch_begin("cross_join_tc", st);
        const cudaError_t e = launch_pdl(kern, dim3(rows.heads(), 64 * KB * 8 * VB / own), dim3(256), 0, st, rec, S, z, image, centre,
                                         S_out, z_out, rows, chunk, ctas, s.Dk, s.Dv);
        const cudaError_t e2 = launch_end("cross_join_tc", st);
        return e != cudaSuccess ? e : e2;
    };
#define LA_MODES(KB, VB, lanes)                                                        \
    (mode == kState     ? go(cross_join_tc<KB, VB, lanes, kState>, 256 / (lanes))      \
     : mode == kCentred ? go(cross_join_tc<KB, VB, lanes, kCentred>, 256 / (lanes))    \
                        : go(cross_join_tc<KB, VB, lanes, kGradSums>, 256 / (lanes)))
    switch (2 * KB + VB) {
        case 3: return many ? LA_MODES(1, 1, 8) : LA_MODES(1, 1, 1);
        case 4: return many ? LA_MODES(1, 2, 8) : LA_MODES(1, 2, 1);
        case 5: return many ? LA_MODES(2, 1, 8) : LA_MODES(2, 1, 1);
        default: return many ? LA_MODES(2, 2, 8) : LA_MODES(2, 2, 1);
    }
#undef LA_MODES
}

cudaError_t tc_fwd(const FwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st) {
    const TcLayout l = tc_layout(s, LA_OP_CROSS_FWD);
    const Rows keys = key_rows(s, a.lens);
    float* rec = reinterpret_cast<float*>(ws);
    CR_TRY(tc_sums(a.k, a.v, keys, rec, l.sum_ctas, s, st));
    CR_TRY(tc_join(kState, rec, nullptr, nullptr, ws + l.S, nullptr, a.S, a.z, keys, kSumRows, l.sum_ctas, s, st));
    return s.N == 0 ? cudaSuccess : answers(a.q, a.o, ws + l.S, false, s, st);
}

cudaError_t tc_apply(const void* q, const float* S, const float* z, void* o, const la_cross_shape& s, char* ws, cudaStream_t st) {
    CR_TRY(tc_join(kState, nullptr, S, z, ws, nullptr, nullptr, nullptr, grouped_queries(s), kRowChunk, 1, s, st));
    return answers(q, o, ws, true, s, st);
}

}  // namespace cross
}  // namespace la
