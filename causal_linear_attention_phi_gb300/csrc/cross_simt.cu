// cross_simt.cu -- CUDA-core kernels of cross attention, forward and gradient (fp32 inputs: one bf16 or tf32 copy of an
// operand is not exact enough; three bf16 parts and six products would be, and are not built).  Chunks of 64 rows; 256 threads seen as 16 x 16 (ty, tx), each with a register tile
// of the chunk's product; operands are fp32 tiles in shared memory read in 16-byte vectors (rows broadcast, columns
// 4 tx + 64 j conflict-free).  Sums are fp32; records of a head are added up in a fixed order.
#include "cross.cuh"
#include "norm_common.cuh"
#include "shared_memory.cuh"

namespace la {
namespace cross {
namespace {

constexpr int kChunk = 64, kThreads = 256;

// Column x of thread tx's W: quads of 4 at 64 j + 4 tx for W >= 4, else W neighbours.
template <int W>
__device__ __forceinline__ int col_of(int tx, int x) {
    return W >= 4 ? 64 * (x >> 2) + 4 * tx + (x & 3) : W * tx + x;
}
template <int W>
__device__ __forceinline__ void load_cols(const float* row, int tx, float (&v)[W]) {
    if constexpr (W >= 4) {
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
            const float4 f = *reinterpret_cast<const float4*>(row + 64 * j + 4 * tx);
            v[4 * j] = f.x, v[4 * j + 1] = f.y, v[4 * j + 2] = f.z, v[4 * j + 3] = f.w;
        }
    } else if constexpr (W == 2) {
        const float2 f = *reinterpret_cast<const float2*>(row + 2 * tx);
        v[0] = f.x, v[1] = f.y;
    } else {
        v[0] = row[tx];
    }
}
template <int W>
__device__ __forceinline__ void store_cols(float* row, int tx, const float (&v)[W]) {
    if constexpr (W >= 4) {
#pragma unroll
        for (int j = 0; j < W / 4; ++j)
            *reinterpret_cast<float4*>(row + 64 * j + 4 * tx) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
#pragma unroll
        for (int x = 0; x < W; ++x) row[W * tx + x] = v[x];
    }
}

// Rows [0, n) of a chunk (phi applied if asked), the rest of its 64 rows 0.  src: the chunk's first row.
template <int D, bool kPhi>
__device__ __forceinline__ void load_rows(float* dst, const float* __restrict__ src, int n) {
#pragma unroll 4
    for (int x = threadIdx.x; x < kChunk * D / 4; x += kThreads) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (4 * x < n * D) {
            f = reinterpret_cast<const float4*>(src)[x];
            if (kPhi) f = make_float4(phi_of(f.x), phi_of(f.y), phi_of(f.z), phi_of(f.w));
        }
        reinterpret_cast<float4*>(dst)[x] = f;
    }
}

// acc[] += x y[]: two columns to an instruction where there are two.
template <int W>
__device__ __forceinline__ void axpy(float x, const float (&y)[W], float (&acc)[W]) {
    if constexpr (W % 2 == 0) {
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            const float2 d = norm::fma2(norm::both(x), make_float2(y[j], y[j + 1]), make_float2(acc[j], acc[j + 1]));
            acc[j] = d.x, acc[j + 1] = d.y;
        }
    } else {
        acc[0] = fmaf(x, y[0], acc[0]);
    }
}
// acc[DA/16][DB/16] += A^T B over the 64 rows of two tiles: rows of acc follow col_of over ty.
template <int DA, int DB>
__device__ __forceinline__ void outer_sum(const float* a, const float* b, float (&acc)[DA / 16][DB / 16], int ty, int tx) {
#pragma unroll 2
    for (int p = 0; p < kChunk; ++p) {
        float x[DA / 16], y[DB / 16];
        load_cols<DA / 16>(a + p * DA, ty, x);
        load_cols<DB / 16>(b + p * DB, tx, y);
#pragma unroll
        for (int i = 0; i < DA / 16; ++i) axpy(x[i], y, acc[i]);
    }
}
// out[4][DB/16] = rows 4 ty .. 4 ty + 3 of A [64][DA] times B [DA][DB].
template <int DA, int DB>
__device__ __forceinline__ void rows_times(const float* a, const float* b, float (&out)[4][DB / 16], int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < DB / 16; ++j) out[i][j] = 0.f;
#pragma unroll 2
    for (int d = 0; d < DA; d += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * DA + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y[DB / 16];
            load_cols<DB / 16>(b + (d + e) * DB, tx, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) axpy(e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w, y, out[i]);
        }
    }
}
template <int DA, int DB>
__device__ __forceinline__ void clear(float (&acc)[DA / 16][DB / 16]) {
#pragma unroll
    for (int i = 0; i < DA / 16; ++i)
#pragma unroll
        for (int j = 0; j < DB / 16; ++j) acc[i][j] = 0.f;
}
// A record: [DK][DV] of the register tiles, then [DK] of threads 0 .. DK - 1.
template <int DK, int DV>
__device__ __forceinline__ void write_record(float* rec, const float (&acc)[DK / 16][DV / 16], float z, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < DK / 16; ++i) store_cols<DV / 16>(rec + col_of<DK / 16>(ty, i) * DV, tx, acc[i]);
    if (threadIdx.x < DK) rec[DK * DV + threadIdx.x] = z;
}
// One thread's running sums take kPeriod chunks of a head, row after row; a block's record takes such periods, each added to what
// it holds (each element by the thread that wrote it) and the sums begun again.  (One sum of 131,072 rows was 5.6e-6 off, of which
// the gradient's differences make more.  B=20 H=16 N=M=4096 128 x 128, one block to a head: 2220 us forward with periods of 8 chunks,
// 2260 of 4, 2190 of all.)
constexpr int kPeriod = 8;
template <int DK, int DV>
__device__ __forceinline__ void close_period(float* rec, float (&acc)[DK / 16][DV / 16], float& z, bool begun, int ty, int tx) {
    if (begun) {
#pragma unroll
        for (int i = 0; i < DK / 16; ++i) {
            float was[DV / 16];
            load_cols<DV / 16>(rec + col_of<DK / 16>(ty, i) * DV, tx, was);
#pragma unroll
            for (int j = 0; j < DV / 16; ++j) acc[i][j] += was[j];
        }
        if (threadIdx.x < DK) z += rec[DK * DV + threadIdx.x];
    }
    write_record<DK, DV>(rec, acc, z, ty, tx);
    clear<DK, DV>(acc);
    z = 0.f;
}

__device__ __forceinline__ Span shared_span(const Rows& r, int chunk, bool dead) {
    __shared__ Span span;
    if (threadIdx.x < 32) {
        const Span s = span_of(r, chunk, dead, blockIdx.x, gridDim.x);
        if (threadIdx.x == 0) span = s;
    }
    __syncthreads();
    return span;
}

// ------------------------------------------------------------------ sums over the keys
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads)
cross_sums_kernel(const float* __restrict__ k, const float* __restrict__ v, float* rec, Rows keys, int slots) {
    extern __shared__ __align__(16) float sm[];
    float *ks = sm, *vs = sm + kChunk * DK;
    pdl_enter();  // launched with programmatic dependent launch
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[DK / 16][DV / 16], z = 0.f;
    clear<DK, DV>(acc);
    Walk w(keys, kChunk, shared_span(keys, kChunk, false));
    bool begun = false;  // the record holds periods of this head
    while (w.more()) {
        const int bh = w.bh;
        bool last;
        int in = 0;
        do {
            const size_t row = (size_t)bh * keys.M + w.row0();
            LA_DCHECK(bh < keys.heads() && w.row0() + w.rows() <= keys.M && w.rows() > 0);
            __syncthreads();
            load_rows<DK, true>(ks, k + row * DK, w.rows());
            load_rows<DV, false>(vs, v + row * DV, w.rows());
            __syncthreads();
            outer_sum<DK, DV>(ks, vs, acc, ty, tx);
            if (threadIdx.x < DK)
                for (int p = 0; p < kChunk; ++p) z += ks[p * DK + threadIdx.x];
            last = w.last();
            w.next();
        } while (++in < kPeriod && !last);
        if (LA_DCHECK((int)blockIdx.x + bh < slots))
            close_period<DK, DV>(rec + (size_t)(blockIdx.x + bh) * (DK * DV + DK), acc, z, begun, ty, tx);
        begun = !last;
    }
}

// ------------------------------------------------------------------ a head's records added up
// E = Dk Dv + Dk floats to a record, the state's first; S and z get their parts.  kLanes threads share four floats, each taking
// every kLanes-th record; their sums are added in a fixed order.
template <int kLanes>
__global__ void __launch_bounds__(256)
cross_join_kernel(const float* __restrict__ rec, float* __restrict__ S, float* __restrict__ z, Rows rows, int chunk,
                  int ctas, int state, int dk) {
    constexpr int kOwn = 256 / kLanes;
    __shared__ float4 part[kLanes][kOwn];
    pdl_enter();  // launched with programmatic dependent launch
    const int bh = blockIdx.x, x = threadIdx.x % kOwn, lane = threadIdx.x / kOwn, E = state + dk, e4 = (blockIdx.y * kOwn + x) * 4;
    const Range g = records_of(rows, chunk, bh, ctas);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e4 < E) {
#pragma unroll 8
        for (int c = g.first + lane; c <= g.last; c += kLanes) {
            const float4 f = *reinterpret_cast<const float4*>(rec + (size_t)(c + bh) * E + e4);
            a.x += f.x, a.y += f.y, a.z += f.z, a.w += f.w;
        }
    }
    if (kLanes > 1) {
        part[lane][x] = a;
        __syncthreads();
        if (lane != 0) return;
#pragma unroll
        for (int l = 1; l < kLanes; ++l) {
            const float4 f = part[l][x];
            a.x += f.x, a.y += f.y, a.z += f.z, a.w += f.w;
        }
    }
    if (e4 >= E) return;
    float* to = e4 < state ? S + (size_t)bh * state + e4 : z + (size_t)bh * dk + (e4 - state);
    *reinterpret_cast<float4*>(to) = a;
}

// ------------------------------------------------------------------ queries
// den of the 64 rows (4 threads to a row) as its inverse
template <int DK>
__device__ __forceinline__ void inverses(const float* ph, const float* zs, float* inv) {
    const int r = threadIdx.x >> 2, part = threadIdx.x & 3;
    float den = 0.f;
#pragma unroll 4
    for (int d = part; d < DK; d += 4) den = fmaf(ph[r * DK + d], zs[d], den);
    den += __shfl_xor_sync(0xffffffffu, den, 1);
    den += __shfl_xor_sync(0xffffffffu, den, 2);
    if (part == 0) inv[r] = over(den);
}

// z of a head to shared memory; whether it has keys.  The whole block.
template <int DK>
__device__ __forceinline__ bool load_z(float* zs, const float* __restrict__ z) {
    const float own = threadIdx.x < DK ? z[threadIdx.x] : 0.f;
    if (threadIdx.x < DK) zs[threadIdx.x] = own;
    return __syncthreads_or(own != 0.f);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads)
cross_apply_kernel(const float* __restrict__ q, const float* __restrict__ S, const float* __restrict__ z, float* __restrict__ o,
                   Rows rows) {
    extern __shared__ __align__(16) float sm[];
    float *Ss = sm, *ph = Ss + DK * DV, *zs = ph + kChunk * DK, *inv = zs + DK;
    pdl_enter();  // launched with programmatic dependent launch
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    bool first = true, alive = false;
    for (Walk w(rows, kChunk, shared_span(rows, kChunk, false)); w.more(); w.next()) {
        __syncthreads();
        if (first || w.fresh) {
            first = false;
            for (int x = threadIdx.x; x < DK * DV / 4; x += kThreads)
                reinterpret_cast<float4*>(Ss)[x] = reinterpret_cast<const float4*>(S + (size_t)w.bh * DK * DV)[x];
            alive = load_z<DK>(zs, z + (size_t)w.bh * DK);
        }
        const size_t row = (size_t)w.bh * rows.M + w.row0();
        LA_DCHECK(w.bh < rows.heads() && w.row0() + w.rows() <= rows.M && w.rows() > 0);
        load_rows<DK, true>(ph, q + row * DK, w.rows());
        __syncthreads();
        inverses<DK>(ph, zs, inv);
        float out[4][DV / 16];
        rows_times<DK, DV>(ph, Ss, out, ty, tx);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            if (r >= w.rows()) break;
#pragma unroll
            for (int j = 0; j < DV / 16; ++j) out[i][j] = alive ? out[i][j] * inv[r] : 0.f;
            store_cols<DV / 16>(o + (row + r) * DV, tx, out[i]);
        }
    }
}

// Heads whose keys and queries are one chunk each: a block forms the head's state in shared memory, where its queries find it.
// One launch and no workspace instead of three launches, which small calls are made of, and no records (in a CUDA graph, B=1 H=2
// N=17 M=64 16 x 16: 6.8 us of three kernels, 3.1 so; 64 x 16 heads of N=M=64 128 x 128: 186 and 171; 256 x 16 of 64 x 64: 312
// and 155); with more chunks to a head the other kernels share them out.
constexpr size_t head_smem(int DK, int DV) { return (size_t)(DK * DV + DK + kChunk + kChunk * (2 * DK + DV)) * 4; }
inline bool one_chunk(const la_cross_shape& s) { return s.M <= kChunk && query_rows(s) <= kChunk; }

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads)
cross_head_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v, float* __restrict__ o,
                  float* __restrict__ S, float* __restrict__ z, Rows keys, int queries) {
    extern __shared__ __align__(16) float sm[];
    float *Ss = sm, *zs = Ss + DK * DV, *inv = zs + DK, *ph = inv + kChunk, *ks = ph + kChunk * DK, *vs = ks + kChunk * DK;
    pdl_enter();  // launched with programmatic dependent launch
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, n = keys.live(blockIdx.x / keys.Hk);
    const size_t key = (size_t)blockIdx.x * keys.M, row = (size_t)blockIdx.x * queries;
    LA_DCHECK(n <= kChunk && queries <= kChunk);
    load_rows<DK, true>(ks, k + key * DK, n);
    load_rows<DV, false>(vs, v + key * DV, n);
    load_rows<DK, true>(ph, q + row * DK, queries);
    __syncthreads();
    float acc[DK / 16][DV / 16], zc = 0.f;
    clear<DK, DV>(acc);
    outer_sum<DK, DV>(ks, vs, acc, ty, tx);
    if (threadIdx.x < DK)
        for (int p = 0; p < kChunk; ++p) zc += ks[p * DK + threadIdx.x];
    write_record<DK, DV>(Ss, acc, zc, ty, tx);  // S, and z behind it
    const bool alive = __syncthreads_or(zc != 0.f);
    if (S) {
        for (int x = threadIdx.x; x < DK * DV / 4; x += kThreads)
            reinterpret_cast<float4*>(S + (size_t)blockIdx.x * DK * DV)[x] = reinterpret_cast<const float4*>(Ss)[x];
        if (threadIdx.x < DK) z[(size_t)blockIdx.x * DK + threadIdx.x] = zs[threadIdx.x];
    }
    if (queries == 0) return;
    inverses<DK>(ph, zs, inv);
    float out[4][DV / 16];
    rows_times<DK, DV>(ph, Ss, out, ty, tx);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= queries) break;
#pragma unroll
        for (int j = 0; j < DV / 16; ++j) out[i][j] = alive ? out[i][j] * inv[r] : 0.f;
        store_cols<DV / 16>(o + (row + r) * DV, tx, out[i]);
    }
}

// dq and the head's records of (R, r).
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads)
cross_query_kernel(const float* __restrict__ q, const float* __restrict__ dout, const float* __restrict__ S,
                   const float* __restrict__ z, float* __restrict__ dq, float* rec, Rows rows, int slots) {
    extern __shared__ __align__(16) float sm[];
    float *St = sm, *ph = St + DK * DV, *ds = ph + kChunk * DK, *zs = ds + kChunk * DV, *inv = zs + DK, *wr = inv + kChunk;
    pdl_enter();  // launched with programmatic dependent launch
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float R[DK / 16][DV / 16], rz = 0.f;
    clear<DK, DV>(R);
    int in = 0;  // chunks of the period so far
    bool first = true, alive = false, begun = false;  // begun: the record holds periods of this head
    for (Walk w(rows, kChunk, shared_span(rows, kChunk, false)); w.more(); w.next()) {
        __syncthreads();
        if (first || w.fresh) {
            first = false;
            for (int x = threadIdx.x; x < DK * DV; x += kThreads)
                St[x] = S[(size_t)w.bh * DK * DV + (x % DK) * DV + x / DK];  // transposed: [dv][dk]
            alive = load_z<DK>(zs, z + (size_t)w.bh * DK);
        }
        const size_t row = (size_t)w.bh * rows.M + w.row0();
        LA_DCHECK(w.bh < rows.heads() && w.row0() + w.rows() <= rows.M && w.rows() > 0);
        load_rows<DK, true>(ph, q + row * DK, w.rows());
        load_rows<DV, false>(ds, dout + row * DV, w.rows());
        __syncthreads();
        inverses<DK>(ph, zs, inv);
        __syncthreads();
        float Y[4][DK / 16];
        rows_times<DV, DK>(ds, St, Y, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            float p[DK / 16], zc[DK / 16], t = 0.f;
            load_cols<DK / 16>(ph + r * DK, tx, p);
            load_cols<DK / 16>(zs, tx, zc);
#pragma unroll
            for (int j = 0; j < DK / 16; ++j) {
                t = fmaf(p[j], Y[i][j] * inv[r], t);
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);  // over the 16 threads of the row
            if (tx == 0) wr[r] = -t;
#pragma unroll
            for (int j = 0; j < DK / 16; ++j)   // t / den could overflow
                Y[i][j] = alive ? fmaf(-t, zc[j], Y[i][j]) * (inv[r] * slope_of(p[j])) : 0.f;
            if (r < w.rows()) store_cols<DK / 16>(dq + (row + r) * DK, tx, Y[i]);
        }
        __syncthreads();
        for (int x = threadIdx.x; x < kChunk * DK; x += kThreads) ph[x] *= inv[x / DK];
        __syncthreads();
        outer_sum<DK, DV>(ph, ds, R, ty, tx);
        if (threadIdx.x < DK)
            for (int p = 0; p < kChunk; ++p) rz = fmaf(ph[p * DK + threadIdx.x], wr[p], rz);
        if (++in < kPeriod && !w.last()) continue;
        if (LA_DCHECK((int)blockIdx.x + w.bh < slots))
            close_period<DK, DV>(rec + (size_t)(blockIdx.x + w.bh) * (DK * DV + DK), R, rz, begun, ty, tx);
        in = 0;
        begun = !w.last();
    }
}

// ------------------------------------------------------------------ gradients of the keys
// `bytes` zero bytes, 16-byte aligned.
__device__ __forceinline__ void zero_bytes(void* p, size_t bytes, int tid, int threads) {
    for (size_t x = tid; x < bytes / 16; x += threads) reinterpret_cast<uint4*>(p)[x] = make_uint4(0u, 0u, 0u, 0u);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads)
cross_key_kernel(const float* __restrict__ k, const float* __restrict__ v, const float* __restrict__ R, const float* __restrict__ rz,
                 float* __restrict__ dk, float* __restrict__ dv, Rows keys) {
    extern __shared__ __align__(16) float sm[];
    float *Rs = sm, *Rt = Rs + DK * DV, *ks = Rt + DK * DV, *vs = ks + kChunk * DK, *rs = vs + kChunk * DV;
    pdl_enter();  // launched with programmatic dependent launch
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    bool first = true;
    for (Walk w(keys, kChunk, shared_span(keys, kChunk, false)); w.more(); w.next()) {
        __syncthreads();
        if (first || w.fresh) {
            first = false;
            for (int x = threadIdx.x; x < DK * DV; x += kThreads) {
                const float f = R[(size_t)w.bh * DK * DV + x];
                Rs[x] = f;
                Rt[(x % DV) * DK + x / DV] = f;
            }
            if (threadIdx.x < DK) rs[threadIdx.x] = rz[(size_t)w.bh * DK + threadIdx.x];
        }
        const size_t row = (size_t)w.bh * keys.M + w.row0();
        LA_DCHECK(w.bh < keys.heads() && w.row0() + w.rows() <= keys.M && w.rows() > 0);
        load_rows<DK, true>(ks, k + row * DK, w.rows());
        load_rows<DV, false>(vs, v + row * DV, w.rows());
        __syncthreads();
        float out[4][DK / 16], ov[4][DV / 16], rc[DK / 16];
        rows_times<DV, DK>(vs, Rt, out, ty, tx);
        rows_times<DK, DV>(ks, Rs, ov, ty, tx);
        load_cols<DK / 16>(rs, tx, rc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            float p[DK / 16];
            load_cols<DK / 16>(ks + r * DK, tx, p);
#pragma unroll
            for (int j = 0; j < DK / 16; ++j) out[i][j] = (out[i][j] + rc[j]) * slope_of(p[j]);
            if (r < w.rows()) {
                store_cols<DK / 16>(dk + (row + r) * DK, tx, out[i]);
                store_cols<DV / 16>(dv + (row + r) * DV, tx, ov[i]);
            }
        }
    }
}

// The rows behind the lengths, [live, M) of every head; a row has k_bytes or v_bytes.
__global__ void __launch_bounds__(256)
cross_clear_kernel(char* __restrict__ dk, char* __restrict__ dv, Rows keys, int k_bytes, int v_bytes) {
    pdl_enter();  // launched with programmatic dependent launch
    const int bh = blockIdx.y, live = keys.live(bh / keys.Hk);
    const size_t row = (size_t)bh * keys.M + live, n = keys.M - live;
    const int tid = blockIdx.x * 256 + threadIdx.x, all = gridDim.x * 256;
    zero_bytes(dk + row * k_bytes, n * k_bytes, tid, all);
    zero_bytes(dv + row * v_bytes, n * v_bytes, tid, all);
}

// ------------------------------------------------------------------ host
// Blocks: a wave of the SMs or two, or one to a chunk.
int blocks_for(long long heads, long long rows, int per_sm) {
    const long long chunks = heads * ((rows + kChunk - 1) / kChunk), most = (long long)kSms * per_sm;
    return (int)(chunks < most ? chunks : most);
}
int key_blocks(const la_cross_shape& s) { return blocks_for((long long)s.B * s.Hk, s.M, 2); }
int query_blocks(const la_cross_shape& s) { return blocks_for((long long)s.B * s.Hk, query_rows(s), 1); }

struct Layout {
    size_t rec, S, z, R, r, bytes;
};
Layout layout(const la_cross_shape& s, bool bwd) {
    const size_t heads = (size_t)s.B * s.Hk, E = (size_t)s.Dk * s.Dv + s.Dk;
    Layout l{};
    size_t blocks = key_blocks(s);
    if (bwd && (size_t)query_blocks(s) > blocks) blocks = query_blocks(s);
    l.S = up((blocks + heads) * E * 4);  // the records first
    l.z = l.S + up(heads * s.Dk * s.Dv * 4);
    l.bytes = l.z + up(heads * s.Dk * 4);
    if (bwd) {
        l.R = l.bytes;
        l.r = l.R + up(heads * s.Dk * s.Dv * 4);
        l.bytes = l.r + up(heads * s.Dk * 4);
    }
    return l;
}

template <typename K, typename... A>
cudaError_t run(const char* name, K kern, dim3 grid, size_t smem, cudaStream_t st, A... args) {
    cudaError_t e = allow_smem(kern, smem);  // a kernel always takes the same
    if (e != cudaSuccess) return e;
    launch_begin(name, st);
    e = launch_pdl(kern, grid, dim3(kThreads), smem, st, args...);
    const cudaError_t e2 = launch_end(name, st);
    return e != cudaSuccess ? e : e2;
}

cudaError_t join(const float* rec, float* S, float* z, const Rows& rows, int ctas, const la_cross_shape& s, cudaStream_t st) {
    const int E = s.Dk * s.Dv + s.Dk;
    auto go = [&](auto kern, int own) {
        return run("cross_join", kern, dim3(rows.heads(), (E + 4 * own - 1) / (4 * own)), 0, st, rec, S, z, rows, kChunk, ctas,
                   s.Dk * s.Dv, s.Dk);
    };
    // forward of N = M = 65536 / heads with one lane and with eight, us: 64 x 64, 2 heads 81 and 71, 8 73 and 71, 16 71 and 79, 48 71 and
    // 78; 128 x 128, 2 heads 160 and 149, 8 150 and 150, 16 149 and 152, 48 152 and 160
    return ctas > 24 * rows.heads() ? go(cross_join_kernel<8>, 32) : go(cross_join_kernel<1>, 256);
}

template <int DK, int DV>
cudaError_t sums(const void* k, const void* v, const Rows& keys, float* rec, float* S, float* z, const la_cross_shape& s,
                 cudaStream_t st) {
    const int ctas = key_blocks(s);
    CR_TRY(run("cross_sums", cross_sums_kernel<DK, DV>, dim3(ctas), kChunk * (DK + DV) * 4, st, (const float*)k, (const float*)v, rec,
               keys, ctas + keys.heads()));
    return join(rec, S, z, keys, ctas, s, st);
}

template <int DK, int DV>
cudaError_t apply(const void* q, const float* S, const float* z, void* o, const la_cross_shape& s, cudaStream_t st) {
    const Rows rows = grouped_queries(s);
    return run("cross_apply", cross_apply_kernel<DK, DV>, dim3(blocks_for(rows.heads(), rows.M, 2)),
               (DK * DV + kChunk * DK + DK + kChunk) * 4, st, (const float*)q, S, z, (float*)o, rows);
}

template <int DK, int DV>
cudaError_t fwd_t(const FwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st) {
    if (one_chunk(s))
        return run("cross_head", cross_head_kernel<DK, DV>, dim3(s.B * s.Hk), head_smem(DK, DV), st, (const float*)a.q, (const float*)a.k,
                   (const float*)a.v, (float*)a.o, a.S, a.z, key_rows(s, a.lens), (int)query_rows(s));
    const Layout l = layout(s, false);
    float *S = a.S ? a.S : reinterpret_cast<float*>(ws + l.S), *z = a.z ? a.z : reinterpret_cast<float*>(ws + l.z);
    CR_TRY((sums<DK, DV>(a.k, a.v, key_rows(s, a.lens), reinterpret_cast<float*>(ws), S, z, s, st)));
    if (s.N == 0) return cudaSuccess;
    return apply<DK, DV>(a.q, S, z, a.o, s, st);
}

template <int DK, int DV>
cudaError_t bwd_t(const BwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st) {
    const Layout l = layout(s, true);
    const Rows keys = key_rows(s, a.lens), rows = grouped_queries(s);
    float *rec = reinterpret_cast<float*>(ws), *R = reinterpret_cast<float*>(ws + l.R), *r = reinterpret_cast<float*>(ws + l.r);
    const float *S = a.S, *z = a.z;
    if (!S) {
        float *Sw = reinterpret_cast<float*>(ws + l.S), *zw = reinterpret_cast<float*>(ws + l.z);
        CR_TRY((sums<DK, DV>(a.k, a.v, keys, rec, Sw, zw, s, st)));
        S = Sw, z = zw;
    }
    const int qc = query_blocks(s);
    CR_TRY(run("cross_query", cross_query_kernel<DK, DV>, dim3(qc), (DK * DV + kChunk * (DK + DV) + DK + 2 * kChunk) * 4, st,
               (const float*)a.q, (const float*)a.dout, S, z, (float*)a.dq, rec, rows, qc + rows.heads()));
    CR_TRY(join(rec, R, r, rows, qc, s, st));
    CR_TRY(run("cross_key", cross_key_kernel<DK, DV>, dim3(blocks_for(keys.heads(), s.M, 1)),
               (2 * DK * DV + kChunk * (DK + DV) + DK) * 4, st, (const float*)a.k, (const float*)a.v, R, r, (float*)a.dk, (float*)a.dv, keys));
    if (!a.lens) return cudaSuccess;
    return run("cross_clear", cross_clear_kernel, dim3(8, keys.heads()), 0, st, (char*)a.dk, (char*)a.dv, keys, 4 * s.Dk, 4 * s.Dv);
}

#define LA_SIZES(F) F(16, 16) F(16, 32) F(16, 64) F(16, 128) F(32, 16) F(32, 32) F(32, 64) F(32, 128) \
    F(64, 16) F(64, 32) F(64, 64) F(64, 128) F(128, 16) F(128, 32) F(128, 64) F(128, 128)

}  // namespace

size_t simt_bytes(const la_cross_shape& s, int op) {
    return op == LA_OP_CROSS_FWD && one_chunk(s) ? 0 : layout(s, op == LA_OP_CROSS_BWD).bytes;
}

cudaError_t simt_fwd(const FwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st) {
#define LA_GO(x, y) \
    if (s.Dk == x && s.Dv == y) return fwd_t<x, y>(a, s, ws, st);
    LA_SIZES(LA_GO)
#undef LA_GO
    return cudaErrorInvalidValue;
}
cudaError_t simt_bwd(const BwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st) {
#define LA_GO(x, y) \
    if (s.Dk == x && s.Dv == y) return bwd_t<x, y>(a, s, ws, st);
    LA_SIZES(LA_GO)
#undef LA_GO
    return cudaErrorInvalidValue;
}
cudaError_t simt_apply(const void* q, const float* S, const float* z, void* o, const la_cross_shape& s, cudaStream_t st) {
#define LA_GO(x, y) \
    if (s.Dk == x && s.Dv == y) return apply<x, y>(q, S, z, o, s, st);
    LA_SIZES(LA_GO)
#undef LA_GO
    return cudaErrorInvalidValue;
}

}  // namespace cross
}  // namespace la
