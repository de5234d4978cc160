// block_norm.cu -- the norms around a block, with its gate and its residual scale.
//   gated norm      y[b,n,h,:] = norm(o[b,h,n,:]) w silu(gate[b,n,h,:])        (heads merged on the way out)
//   residual norm   h = x + scale a,  y = norm(h) w + b
// norm(x) = (x - mean) rstd, or x rstd with rstd = 1 / sqrt(mean x^2 + eps).  With n = norm(x) and d = dL/dn,
//   dL/dx = rstd (d - n mean(d n) - mean(d)), the last term for the layer norm only.
// Bound by memory: every array is read once and written once; statistics, sums and products are fp32 and each output is
// rounded once, from the unrounded values (y is formed from the unrounded h).  Sums over rows are kept in registers by
// column, written once to a block and added up by a second kernel in a fixed order: the same bits every time.
#include "block_norm.cuh"
#include "norm_common.cuh"
#include "shared_memory.cuh"

namespace la {
namespace bn {
namespace {

using namespace norm;

// A 16-byte vector as floats, and back.
template <typename T>
struct Vec {
    static constexpr int n = 16 / (int)sizeof(T);
    __device__ static void get(const uint4& w, float (&v)[n]) {
        float2 p[n / 2];
        Pairs<T>::get(&w, p);
#pragma unroll
        for (int e = 0; e < n / 2; ++e) v[2 * e] = p[e].x, v[2 * e + 1] = p[e].y;
    }
    __device__ static void load(const void* p, float (&v)[n]) { get(*reinterpret_cast<const uint4*>(p), v); }
    __device__ static void put(void* to, const float (&v)[n]) {
        float2 p[n / 2];
#pragma unroll
        for (int e = 0; e < n / 2; ++e) p[e] = make_float2(v[2 * e], v[2 * e + 1]);
        Pairs<T>::put(to, p);
    }
};

__device__ __forceinline__ float rcp(float x) {  // 1 ulp
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2_approx(-1.4426950408889634f * x)); }

template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ------------------------------------------------------------------ gated norm
// A row is a head at a position; rows are numbered as the gate has them, position by position.  L lanes own a row, 16 bytes
// each, so the gate's side is contiguous and the heads' side comes in whole rows.  A block takes kU rows to a lane group
// at a time and issues all their loads before any arithmetic.
constexpr int kBlock = 256;
constexpr int kFwdU = 4;
// The gradient of bf16 rows: two rows at a time and four blocks to an SM (four and two: 488 us instead of 435 for B=2 H=16 N=65536
// D=128); fp32 rows, half as long to a lane, are better off with four (203 us instead of 230 for N=16384 D=128).
template <typename T>
constexpr int bwd_u() { return sizeof(T) == 2 ? 2 : 4; }

struct GatedRows {
    long long rows;       // B N H
    int N, H;
    unsigned magic;       // ceil(2^32 / H): x / H = x magic >> 32 for x H < 2^32, H > 1
};

// The head-major row of row f0 + l: f0's (b, n, h) is known, l is small.
struct Place {
    int b, n, h;
    __device__ long long row(const GatedRows& g, int l) const {
        const unsigned x = (unsigned)(h + l), H = g.H, N = g.N;
        const unsigned c = H == 1 ? x : H > 1024 ? (x >= H ? 1u : 0u) : __umulhi(x, g.magic);  // x / H; l < 1024
        unsigned nn = n + c, bb = b;
        if (nn >= N) {
            bb += nn / N;
            nn %= N;
        }
        return ((long long)bb * H + (x - c * H)) * N + nn;
    }
    __device__ static Place of(const GatedRows& g, long long f) {
        const long long p = f / g.H;
        return Place{(int)(p / g.N), (int)(p % g.N), (int)(f - p * g.H)};
    }
};

// norm's statistics of a row held by L lanes: v becomes x - mean; returns rstd.
template <int L, int n>
__device__ __forceinline__ float centre(float2 (&v)[n], float inv_d, bool rms, float eps) {
    if (!rms) {
        float2 s = v[0];
#pragma unroll
        for (int e = 1; e < n; ++e) s = add2(s, v[e]);
        const float2 mu = both(-lanes_sum<L>(s.x + s.y) * inv_d);
#pragma unroll
        for (int e = 0; e < n; ++e) v[e] = add2(v[e], mu);
    }
    float2 s = mul2(v[0], v[0]);
#pragma unroll
    for (int e = 1; e < n; ++e) s = fma2(v[e], v[e], s);
    return 1.f / sqrtf(fmaf(lanes_sum<L>(s.x + s.y), inv_d, eps));
}

template <typename T, int L>
__global__ void __launch_bounds__(kBlock, 4)
gated_fwd_kernel(const T* o, const T* gate, const T* __restrict__ w, T* y, GatedRows g, int rms, float eps) {
    using V = Vec<T>;
    constexpr int kRows = kBlock / L, D = L * V::n, kP = V::n / 2, kU = kFwdU;
    pdl_enter();  // launched with programmatic dependent launch
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    float2 wv[kP];
#pragma unroll
    for (int e = 0; e < kP; ++e) wv[e] = both(1.f);
    if (w) Pairs<T>::get(w + lane * V::n, wv);
    for (long long f0 = (long long)blockIdx.x * (kRows * kU); f0 < g.rows; f0 += (long long)gridDim.x * (kRows * kU)) {
        const Place at = Place::of(g, f0);
        uint4 xo[kU], xg[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int l = u * kRows + sub;
            xo[u] = xg[u] = make_uint4(0u, 0u, 0u, 0u);
            if (f0 + l >= g.rows) continue;
            const long long r = at.row(g, l);
            LA_DCHECK(r >= 0 && r < g.rows);
            xo[u] = *reinterpret_cast<const uint4*>(o + r * D + lane * V::n);
            xg[u] = *reinterpret_cast<const uint4*>(gate + (f0 + l) * D + lane * V::n);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int l = u * kRows + sub;
            float2 v[kP];
            float x[V::n], s[V::n];
            Pairs<T>::get(&xo[u], v);
            V::get(xg[u], s);
            const float rs = centre<L>(v, 1.f / D, rms, eps);
#pragma unroll
            for (int e = 0; e < V::n; ++e) {
                const float n = (e & 1 ? v[e >> 1].y : v[e >> 1].x) * rs, wt = e & 1 ? wv[e >> 1].y : wv[e >> 1].x;
                x[e] = n * wt * (s[e] * sigmoid(s[e]));
            }
            if (f0 + l < g.rows) V::put(y + (f0 + l) * D + lane * V::n, x);
        }
    }
}

// part: [blocks][D]
template <typename T, int L>
__global__ void __launch_bounds__(kBlock, sizeof(T) == 2 ? 4 : 2)
gated_bwd_kernel(const T* o, const T* gate, const T* __restrict__ w, const T* dy, T* dout, T* dgate,
                 float* __restrict__ part, GatedRows g, int rms, float eps) {
    using V = Vec<T>;
    constexpr int kRows = kBlock / L, D = L * V::n, kP = V::n / 2, kU = bwd_u<T>();
    __shared__ __align__(16) float sums[kRows][D];
    pdl_enter();  // launched with programmatic dependent launch
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    float2 wv[kP], dw[kP];
#pragma unroll
    for (int e = 0; e < kP; ++e) wv[e] = both(1.f), dw[e] = both(0.f);
    if (w) Pairs<T>::get(w + lane * V::n, wv);
    for (long long f0 = (long long)blockIdx.x * (kRows * kU); f0 < g.rows; f0 += (long long)gridDim.x * (kRows * kU)) {
        const Place at = Place::of(g, f0);
        uint4 xo[kU], xg[kU], xd[kU];
        long long r[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int l = u * kRows + sub;
            xo[u] = xg[u] = xd[u] = make_uint4(0u, 0u, 0u, 0u);
            r[u] = 0;
            if (f0 + l >= g.rows) continue;
            r[u] = at.row(g, l);
            LA_DCHECK(r[u] >= 0 && r[u] < g.rows);
            xo[u] = *reinterpret_cast<const uint4*>(o + r[u] * D + lane * V::n);
            xg[u] = *reinterpret_cast<const uint4*>(gate + (f0 + l) * D + lane * V::n);
            xd[u] = *reinterpret_cast<const uint4*>(dy + (f0 + l) * D + lane * V::n);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int l = u * kRows + sub;
            const bool in = f0 + l < g.rows;
            float2 v[kP], s[kP], d[kP];
            Pairs<T>::get(&xo[u], v);
            Pairs<T>::get(&xg[u], s);
            Pairs<T>::get(&xd[u], d);
            const float rstd = centre<L>(v, 1.f / D, rms, eps);  // every lane takes part
            const float rs = in ? rstd : 0.f;                    // rows behind the last add nothing
            float2 m0 = both(0.f), m1 = both(0.f);
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                const float2 t = mul2(s[e], both(-1.4426950408889634f)), q = add2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), both(1.f));
                const float2 sg = make_float2(rcp(q.x), rcp(q.y)), silu = mul2(s[e], sg);
                v[e] = mul2(v[e], both(rs));
                const float2 dn = mul2(d[e], v[e]);  // d(w silu)
                dw[e] = fma2(dn, silu, dw[e]);
                s[e] = mul2(mul2(dn, wv[e]), fma2(silu, fma2(sg, both(-1.f), both(1.f)), sg));  // dgate: silu' = sg + silu (1 - sg)
                d[e] = mul2(d[e], mul2(silu, wv[e]));
                m1 = fma2(d[e], v[e], m1);
                if (!rms) m0 = add2(m0, d[e]);
            }
            const float2 k1 = both(-lanes_sum<L>(m1.x + m1.y) * (1.f / D)), k0 = both(rms ? 0.f : -lanes_sum<L>(m0.x + m0.y) * (1.f / D));
#pragma unroll
            for (int e = 0; e < kP; ++e) d[e] = mul2(both(rs), fma2(v[e], k1, add2(d[e], k0)));
            if (!in) continue;
            Pairs<T>::put(dgate + (f0 + l) * D + lane * V::n, s);
            Pairs<T>::put(dout + r[u] * D + lane * V::n, d);
        }
    }
    if (!part) return;
#pragma unroll
    for (int e = 0; e < kP; ++e) *reinterpret_cast<float2*>(&sums[sub][lane * V::n + 2 * e]) = dw[e];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kBlock) {
        float a = 0.f;
#pragma unroll 8
        for (int x = 0; x < kRows; ++x) a += sums[x][c];
        part[(size_t)blockIdx.x * D + c] = a;
    }
}

// ------------------------------------------------------------------ sums over rows
// out[which][C] = the blocks' records [blocks][which < K][C] (pitch floats apart) added up: 32 columns by 32 lanes of blocks.
struct Outs {
    void* p[3];
};
template <typename T>
__global__ void __launch_bounds__(1024)
columns_join_kernel(const float* __restrict__ part, Outs out, int blocks, int C, int K, int pitch) {
    __shared__ float s[32][33];
    pdl_enter();  // launched with programmatic dependent launch
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx, all = K * C;
    float v = 0.f;
    if (c < all) {
#pragma unroll 10
        for (int i = ty; i < blocks; i += 32) v += part[(size_t)i * pitch + c];  // in that order; the loads of ten go together
    }
    s[ty][tx] = v;
    __syncthreads();
    v = s[tx][ty];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int col = blockIdx.x * 32 + ty;
    if (tx != 0 || col >= all) return;
    T* to = static_cast<T*>(col < C ? out.p[0] : col < 2 * C ? out.p[1] : out.p[2]);
    if (to) to[col % C] = from_f32<T>(v);
}

// ------------------------------------------------------------------ residual norm, rows that 16-byte vectors divide
// Rows are contiguous, so a tile of them is one bulk copy to an array; a block keeps `stages` sets of tiles in flight in
// shared memory.  TPR threads own a row, kBlock (or TPR) / TPR rows at a time, VPT vectors to a thread, always the same columns.
constexpr int kMostStages = 3;
struct Tiles {
    long long rows, tiles;
    int C, R, stages;  // R rows to a tile
    uint32_t row;      // bytes
};

template <int TPR>
constexpr int block_of() { return TPR > kBlock ? TPR : kBlock; }

template <typename T, int VPT, int TPR>
__global__ void __launch_bounds__(block_of<TPR>())
resid_fwd_tiles(const T* x, const T* a, const T* __restrict__ scale, const T* __restrict__ w, const T* __restrict__ b, T* h, T* y,
                float* __restrict__ mean, float* __restrict__ rstd, Tiles tl, int rms, float eps, int* err) {
    using V = Vec<T>;
    constexpr int kRows = block_of<TPR>() / TPR;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bar[kMostStages];
    __shared__ float buf[kRows][2][TPR > 256 ? 16 : 8];
    const int tid = threadIdx.x, t = tid % TPR, sub = tid / TPR, nv = tl.C / V::n, stages = tl.stages;
    const uint32_t tile = tl.row * tl.R;
    if (tid == 0) {
        for (int s = 0; s < kMostStages; ++s) sm100::mbar_init(bar + s, 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();  // launched with programmatic dependent launch
    auto rows_of = [&](long long k) { return (int)min((long long)tl.R, tl.rows - k * tl.R); };
    bool ok = true;
    long long issued = 0;
    auto load = [&](long long i, int s) {  // the i-th tile of this block
        const long long k = blockIdx.x + i * gridDim.x;
        if (tid != 0 || k >= tl.tiles || !ok) return;
        issued = i + 1;
        const uint32_t bytes = rows_of(k) * tl.row;
        LA_DCHECK(bytes <= tile && k * tl.R + rows_of(k) <= tl.rows);
        sm100::mbar_arrive_expect_tx(bar + s, 2 * bytes);
        sm100::bulk_load(smem + (2 * s) * tile, reinterpret_cast<const uint8_t*>(x) + k * tile, bytes, bar + s);
        sm100::bulk_load(smem + (2 * s + 1) * tile, reinterpret_cast<const uint8_t*>(a) + k * tile, bytes, bar + s);
    };
    for (int i = 0; i < stages; ++i) load(i, i);
    const float inv = 1.f / (float)tl.C;
    int turn = 0, s = 0, phase = 0;
    long long i = 0;
    for (long long k = blockIdx.x; k < tl.tiles; k += gridDim.x, ++i) {
        const int n = rows_of(k);
        ok = ok && sm100::mbar_wait(bar + s, phase, err, LA_ERR_TIMEOUT);
        __syncwarp();
        for (int r0 = 0; r0 < n; r0 += kRows) {
            const int r = r0 + sub;
            const bool in = r < n;  // the same for a whole warp where a row has a barrier
            if (TPR > 32 && !in) break;
            const long long row = k * tl.R + (in ? r : 0);
            LA_DCHECK(row < tl.rows);
            const uint8_t* xr = smem + 2 * s * tile + (in ? r : 0) * tl.row;
            const uint8_t* ar = xr + tile;
            uint8_t *hr = reinterpret_cast<uint8_t*>(h) + row * tl.row, *yr = reinterpret_cast<uint8_t*>(y) + row * tl.row;
            float v[VPT][V::n], sum[1] = {0.f};
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = t + TPR * j;
                if (c >= nv) continue;
                float av[V::n], sc[V::n];
                V::load(xr + 16 * c, v[j]);
                V::load(ar + 16 * c, av);
                if (scale) V::load(reinterpret_cast<const uint4*>(scale) + c, sc);
#pragma unroll
                for (int e = 0; e < V::n; ++e) {
                    v[j][e] = scale ? fmaf(sc[e], av[e], v[j][e]) : v[j][e] + av[e];
                    sum[0] += v[j][e];
                }
                if (in) V::put(hr + 16 * c, v[j]);
            }
            float mu = 0.f;
            if (!rms) {
                group_sum<TPR, 1>(sum, buf[sub], sub, t, turn);
                mu = __fmul_rn(sum[0], inv);
            }
            sum[0] = 0.f;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (t + TPR * j < nv)
#pragma unroll
                    for (int e = 0; e < V::n; ++e) {
                        v[j][e] -= mu;
                        sum[0] = fmaf(v[j][e], v[j][e], sum[0]);
                    }
            group_sum<TPR, 1>(sum, buf[sub], sub, t, turn);
            const float rs = 1.f / sqrtf(fmaf(sum[0], inv, eps));
            if (!in) continue;
            if (t == 0) {
                if (mean) mean[row] = mu;
                if (rstd) rstd[row] = rs;
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = t + TPR * j;
                if (c >= nv) continue;
                float wv[V::n], bv[V::n];
                if (w) V::load(reinterpret_cast<const uint4*>(w) + c, wv);
                if (b) V::load(reinterpret_cast<const uint4*>(b) + c, bv);
#pragma unroll
                for (int e = 0; e < V::n; ++e) {
                    v[j][e] = __fmul_rn(v[j][e], rs);
                    v[j][e] = fmaf(v[j][e], w ? wv[e] : 1.f, b ? bv[e] : 0.f);
                }
                V::put(yr + 16 * c, v[j]);
            }
        }
        __syncthreads();  // the tiles have been read
        load(i + stages, s);
        if (++s == stages) s = 0, phase ^= 1;
    }
    if (!ok) sm100::mbar_drain(bar, stages, issued, err, LA_ERR_TIMEOUT);
}

// The arrays of the gradient in a stage: h, dy, then dh and a where there are any.
template <typename T, int VPT, int TPR>
__global__ void __launch_bounds__(block_of<TPR>(), TPR > kBlock ? 1 : 2)
resid_bwd_tiles(const T* h, const T* a, const T* __restrict__ scale, const T* __restrict__ w, const float* __restrict__ mean,
                const float* __restrict__ rstd, const T* dy, const T* dh, T* dx, T* da, float* __restrict__ part, Tiles tl,
                int rms, int* err) {
    using V = Vec<T>;
    constexpr int kThr = block_of<TPR>(), kRows = kThr / TPR, kP = V::n / 2;
    constexpr bool kKeep = VPT * V::n <= 16;  // n and d in registers between the passes, else formed again
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bar[kMostStages];
    __shared__ float buf[kRows][4][TPR > 256 ? 16 : 8];
    const int tid = threadIdx.x, t = tid % TPR, sub = tid / TPR, nv = tl.C / V::n, stages = tl.stages;
    const uint32_t tile = tl.row * tl.R, at_dh = 2 * tile, at_a = at_dh + (dh ? tile : 0), set = at_a + (a ? tile : 0);
    if (tid == 0) {
        for (int s = 0; s < kMostStages; ++s) sm100::mbar_init(bar + s, 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();  // launched with programmatic dependent launch
    auto rows_of = [&](long long k) { return (int)min((long long)tl.R, tl.rows - k * tl.R); };
    bool ok = true;
    long long issued = 0;
    auto load = [&](long long i, int s) {
        const long long k = blockIdx.x + i * gridDim.x;
        if (tid != 0 || k >= tl.tiles || !ok) return;
        issued = i + 1;
        const uint32_t bytes = rows_of(k) * tl.row;
        LA_DCHECK(bytes <= tile && k * tl.R + rows_of(k) <= tl.rows);
        uint8_t* to = smem + s * set;
        sm100::mbar_arrive_expect_tx(bar + s, (set / tile) * bytes);
        sm100::bulk_load(to, reinterpret_cast<const uint8_t*>(h) + k * tile, bytes, bar + s);
        sm100::bulk_load(to + tile, reinterpret_cast<const uint8_t*>(dy) + k * tile, bytes, bar + s);
        if (dh) sm100::bulk_load(to + at_dh, reinterpret_cast<const uint8_t*>(dh) + k * tile, bytes, bar + s);
        if (a) sm100::bulk_load(to + at_a, reinterpret_cast<const uint8_t*>(a) + k * tile, bytes, bar + s);
    };
    for (int i = 0; i < stages; ++i) load(i, i);
    float2 dw[VPT][kP], db[VPT][kP], ds[VPT][kP];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < kP; ++e) dw[j][e] = db[j][e] = ds[j][e] = both(0.f);
    const float inv = 1.f / (float)tl.C;
    float mu_next = 0.f, rs_next = 0.f;  // the statistics of this thread's next row, loaded a turn ahead
    auto stats = [&](long long k, int r) {
        if (k < tl.tiles && r < rows_of(k)) {
            if (!rms) mu_next = mean[k * tl.R + r];
            rs_next = rstd[k * tl.R + r];
        }
    };
    stats(blockIdx.x, sub);
    int turn = 0, s = 0, phase = 0;
    long long i = 0;
    for (long long k = blockIdx.x; k < tl.tiles; k += gridDim.x, ++i) {
        const int n = rows_of(k);
        ok = ok && sm100::mbar_wait(bar + s, phase, err, LA_ERR_TIMEOUT);
        __syncwarp();
        for (int r0 = 0; r0 < n; r0 += kRows) {
            const int r = r0 + sub;
            const bool in = r < n;
            const float mu = mu_next, rs = rs_next;
            if (r0 + kRows < n)
                stats(k, r + kRows);
            else
                stats(k + gridDim.x, sub);
            if (TPR > 32 && !in) break;
            const long long row = k * tl.R + (in ? r : 0);
            LA_DCHECK(row < tl.rows);
            const uint8_t* hr = smem + s * set + (in ? r : 0) * tl.row;
            float2 n[kKeep ? VPT : 1][kP], d[kKeep ? VPT : 1][kP], s0 = both(0.f), s1 = s0;
            auto normed = [&](int j, float2 (&g)[kP]) {  // n and d of vector j, g = dy
                const int c = t + TPR * j, q = kKeep ? j : 0;
                Pairs<T>::get(hr + 16 * c, n[q]);
                Pairs<T>::get(hr + tile + 16 * c, g);
                if (w) Pairs<T>::get(reinterpret_cast<const uint4*>(w) + c, d[q]);
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    n[q][e] = mul2(add2(n[q][e], both(-mu)), both(rs));
                    d[q][e] = w ? mul2(g[e], d[q][e]) : g[e];
                }
            };
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (!in || t + TPR * j >= nv) continue;
                const int q = kKeep ? j : 0;
                float2 g[kP];
                normed(j, g);
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    s0 = add2(s0, d[q][e]);
                    s1 = fma2(d[q][e], n[q][e], s1);
                    dw[j][e] = fma2(g[e], n[q][e], dw[j][e]);
                    db[j][e] = add2(db[j][e], g[e]);
                }
            }
            float sum[2] = {s0.x + s0.y, s1.x + s1.y};
            group_sum<TPR, 2>(sum, buf[sub], sub, t, turn);
            if (!in) continue;
            const float2 m0 = both(rms ? 0.f : -__fmul_rn(sum[0], inv)), m1 = both(-__fmul_rn(sum[1], inv));
            uint8_t *ox = reinterpret_cast<uint8_t*>(dx) + row * tl.row, *oa = reinterpret_cast<uint8_t*>(da) + row * tl.row;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = t + TPR * j, q = kKeep ? j : 0;
                if (c >= nv) continue;
                float2 g[kP], x[kP];
                if (!kKeep) normed(j, g);
                if (dh) Pairs<T>::get(hr + at_dh + 16 * c, x);
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    g[e] = fma2(n[q][e], m1, add2(d[q][e], m0));
                    g[e] = dh ? fma2(both(rs), g[e], x[e]) : mul2(both(rs), g[e]);
                }
                Pairs<T>::put(ox + 16 * c, g);
                if (a) {
                    Pairs<T>::get(hr + at_a + 16 * c, x);
#pragma unroll
                    for (int e = 0; e < kP; ++e) ds[j][e] = fma2(x[e], g[e], ds[j][e]);
                }
                if (da) {
                    if (scale) {
                        Pairs<T>::get(reinterpret_cast<const uint4*>(scale) + c, x);
#pragma unroll
                        for (int e = 0; e < kP; ++e) g[e] = mul2(g[e], x[e]);
                    }
                    Pairs<T>::put(oa + 16 * c, g);
                }
            }
        }
        __syncthreads();  // the tiles have been read
        load(i + stages, s);
        if (++s == stages) s = 0, phase ^= 1;
    }
    if (!ok) sm100::mbar_drain(bar, stages, issued, err, LA_ERR_TIMEOUT);
    if (!part) return;
    // the rows of a block joined in shared memory (the tiles are done with), then one record per block
    float* sums = reinterpret_cast<float*>(smem);
    float* p = part + (size_t)blockIdx.x * 3 * tl.C;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
        if (which == 2 && !a) break;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = t + TPR * j;
            if (c >= nv) continue;
#pragma unroll
            for (int e = 0; e < kP; ++e)
                *reinterpret_cast<float2*>(sums + sub * tl.C + c * V::n + 2 * e) = which == 0 ? dw[j][e] : which == 1 ? db[j][e] : ds[j][e];
        }
        __syncthreads();
        for (int c = tid; c < tl.C; c += kThr) {
            float v = 0.f;
            for (int r = 0; r < kRows; ++r) v += sums[r * tl.C + c];
            p[which * tl.C + c] = v;
        }
    }
}

// ------------------------------------------------------------------ residual norm, other rows: element by element
// Rows go from memory to registers; VPT elements to a thread, TPR threads to a row.
template <typename T, int VPT, int TPR>
__global__ void __launch_bounds__(block_of<TPR>())
resid_fwd_elements(const T* x, const T* a, const T* __restrict__ scale, const T* __restrict__ w, const T* __restrict__ b, T* h,
                   T* y, float* __restrict__ mean, float* __restrict__ rstd, long long rows, int C, int rms, float eps) {
    constexpr int kRows = block_of<TPR>() / TPR;
    __shared__ float buf[kRows][2][TPR > 256 ? 16 : 8];
    pdl_enter();  // launched with programmatic dependent launch
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const float inv = 1.f / (float)C;
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * kRows; r0 < rows; r0 += (long long)gridDim.x * kRows) {
        const bool in = r0 + sub < rows;
        if (TPR > 32 && !in) break;
        const long long at = (in ? r0 + sub : r0) * C;
        float v[VPT], sum[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = t + TPR * j;
            v[j] = 0.f;
            if (c >= C) continue;
            const float av = to_f32(a[at + c]), xv = to_f32(x[at + c]);
            v[j] = scale ? fmaf(to_f32(scale[c]), av, xv) : xv + av;
            sum[0] += v[j];
        }
        float mu = 0.f;
        if (!rms) {
            group_sum<TPR, 1>(sum, buf[sub], sub, t, turn);
            mu = __fmul_rn(sum[0], inv);
        }
        sum[0] = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (t + TPR * j < C) sum[0] = fmaf(v[j] - mu, v[j] - mu, sum[0]);
        group_sum<TPR, 1>(sum, buf[sub], sub, t, turn);
        const float rs = 1.f / sqrtf(fmaf(sum[0], inv, eps));
        if (!in) continue;
        if (t == 0) {
            if (mean) mean[r0 + sub] = mu;
            if (rstd) rstd[r0 + sub] = rs;
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = t + TPR * j;
            if (c >= C || !LA_DCHECK(at + c < rows * C)) continue;
            h[at + c] = from_f32<T>(v[j]);
            y[at + c] = from_f32<T>(fmaf(__fmul_rn(v[j] - mu, rs), w ? to_f32(w[c]) : 1.f, b ? to_f32(b[c]) : 0.f));
        }
    }
}

template <typename T, int VPT, int TPR>
__global__ void __launch_bounds__(block_of<TPR>(), TPR > kBlock ? 1 : 5)
resid_bwd_elements(const T* h, const T* a, const T* __restrict__ scale, const T* __restrict__ w, const float* __restrict__ mean,
                   const float* __restrict__ rstd, const T* dy, const T* dh, T* dx, T* da, float* __restrict__ part,
                   long long rows, int C, int rms) {
    constexpr int kThr = block_of<TPR>(), kRows = kThr / TPR, kAhead = VPT <= 8 ? VPT : 8;
    extern __shared__ float sums[];  // [kRows][C], where a block has several rows
    __shared__ float buf[kRows][4][TPR > 256 ? 16 : 8];
    pdl_enter();  // launched with programmatic dependent launch
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const float inv = 1.f / (float)C;
    float dw[VPT], db[VPT], ds[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) dw[j] = db[j] = ds[j] = 0.f;
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * kRows; r0 < rows; r0 += (long long)gridDim.x * kRows) {
        const bool in = r0 + sub < rows;
        if (TPR > 32 && !in) break;
        const long long row = in ? r0 + sub : r0, at = row * C;
        const float mu = rms ? 0.f : mean[row], rs = rstd[row];
        // what a row needs is loaded together, before any use or store (the outputs may lie in the inputs' arrays)
        float n[VPT], d[VPT], xh[kAhead], xa[kAhead], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const bool here = in && t + TPR * j < C;
            n[j] = here ? to_f32(h[at + t + TPR * j]) : mu;
            d[j] = here ? to_f32(dy[at + t + TPR * j]) : 0.f;
        }
        auto fetch = [&](int j0) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int c = t + TPR * (j0 + j);
                xh[j] = in && c < C && dh ? to_f32(dh[at + c]) : 0.f;
                xa[j] = in && c < C && a ? to_f32(a[at + c]) : 0.f;
            }
        };
        fetch(0);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const float g = d[j];
            n[j] = __fmul_rn(n[j] - mu, rs);
            if (w && t + TPR * j < C) d[j] = __fmul_rn(g, to_f32(w[t + TPR * j]));
            sum[0] += d[j];
            sum[1] = fmaf(d[j], n[j], sum[1]);
            dw[j] = fmaf(g, n[j], dw[j]);
            db[j] += g;
        }
        group_sum<TPR, 2>(sum, buf[sub], sub, t, turn);
        if (!in) continue;
        const float m0 = rms ? 0.f : __fmul_rn(sum[0], inv), m1 = __fmul_rn(sum[1], inv);
#pragma unroll
        for (int j0 = 0; j0 < VPT; j0 += kAhead) {
            if (j0 > 0) fetch(j0);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int j = j0 + k, c = t + TPR * j;
                if (c >= C || !LA_DCHECK(at + c < rows * C)) continue;
                const float g = fmaf(rs, fmaf(-n[j], m1, d[j] - m0), xh[k]);
                ds[j] = fmaf(xa[k], g, ds[j]);
                dx[at + c] = from_f32<T>(g);
                if (da) da[at + c] = from_f32<T>(scale ? to_f32(scale[c]) * g : g);
            }
        }
    }
    if (!part) return;
    float* p = part + (size_t)blockIdx.x * 3 * C;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
        if (which == 2 && !a) break;
        float* to = kRows == 1 ? p + which * C : sums + sub * C;
        if (kRows > 1) __syncthreads();
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (t + TPR * j < C) to[t + TPR * j] = which == 0 ? dw[j] : which == 1 ? db[j] : ds[j];
        if (kRows == 1) continue;
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += kThr) {
            float v = 0.f;
            for (int r = 0; r < kRows; ++r) v += sums[r * C + c];
            p[which * C + c] = v;
        }
    }
}

// ------------------------------------------------------------------ host
template <typename K, typename... A>
cudaError_t run(const char* name, K kern, long long blocks, int block, size_t smem, cudaStream_t st, A... args) {
    launch_begin(name, st);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)blocks), dim3(block), smem, st, args...);
    const cudaError_t e2 = launch_end(name, st);
    return e != cudaSuccess ? e : e2;
}

int elem_of(int dtype) { return dtype == LA_BF16 ? 2 : 4; }

GatedRows rows_of(const Gated& g) {
    GatedRows r{};
    r.rows = g.positions * g.H;
    r.N = g.N;
    r.H = g.H;
    r.magic = (unsigned)((0x100000000ull + g.H - 1) / g.H);
    return r;
}
int gated_blocks(const Gated& g, int u, int per_sm) {
    const long long rows = g.positions * g.H, at_once = (long long)u * kBlock / (g.D * elem_of(g.dtype) / 16);
    const long long tiles = (rows + at_once - 1) / at_once, most = 152LL * per_sm;
    return (int)(tiles < most ? tiles : most);
}
constexpr int kGatedFwdPerSm = 8;
// The gradient's blocks (and records): a wave of the SMs.
int gated_bwd_blocks(const Gated& g) { return g.dtype == LA_BF16 ? gated_blocks(g, bwd_u<__nv_bfloat16>(), 4) : gated_blocks(g, bwd_u<float>(), 2); }

template <typename T, int L>
cudaError_t gated_fwd_l(const void* o, const void* gate, const void* w, void* y, const Gated& g, cudaStream_t st) {
    return run("gated_fwd", gated_fwd_kernel<T, L>, gated_blocks(g, kFwdU, kGatedFwdPerSm), kBlock, 0, st, (const T*)o, (const T*)gate,
               (const T*)w, (T*)y, rows_of(g), g.rms, g.eps);
}
template <typename T, int L>
cudaError_t gated_bwd_l(const void* o, const void* gate, const void* w, const void* dy, void* dout, void* dgate, void* dw,
                        const Gated& g, float* part, cudaStream_t st) {
    const int blocks = gated_bwd_blocks(g);
    const cudaError_t e = run("gated_bwd", gated_bwd_kernel<T, L>, blocks, kBlock, 0, st, (const T*)o, (const T*)gate,
                              (const T*)w, (const T*)dy, (T*)dout, (T*)dgate, part, rows_of(g), g.rms, g.eps);
    if (e != cudaSuccess || !part) return e;
    return run("columns_join", columns_join_kernel<T>, (g.D + 31) / 32, 1024, 0, st, (const float*)part, Outs{{dw, nullptr, nullptr}},
               blocks, g.D, 1, g.D);
}

// Elements to a thread: 8 forward, 16 in the gradient (whose threads hold three sums to an element; 8 took 297 us instead of 267 for
// 65536 x 2048 bf16, where the forward takes 353 us instead of 370 for 131072 x 2048); up to 32 of the widest rows.
constexpr int kFwdElems = 8, kBwdElems = 16;
// Rows that vectors do not divide: 65536 x 1001 bf16 takes 137 us forward with 16 (154 with 8), the gradient 263 us with 4 and five
// blocks to an SM (444 with 8 and three, 820 with 16 and two: its loads wait for one another, so many short rows it is).
constexpr int kFwdSingles = 16, kBwdSingles = 4;
int row_threads(int C, int elems) {
    int t = 8;
    while (t < 512 && t * elems < C) t *= 2;
    return t;
}
int block_for(int threads) { return threads > kBlock ? threads : kBlock; }
bool vectors(int C, int elem) { return C % (16 / elem) == 0; }
constexpr size_t kMostSmem = 225000;
// The gradient's rows go through shared memory where four of them fit (fp32 rows above 14062 elements do not).
bool bwd_streams(const la_norm_shape& s) {
    return vectors(s.C, elem_of(s.dtype)) && (size_t)4 * s.C * elem_of(s.dtype) <= kMostSmem;
}
// A tile of about `bytes` to an array, fewer rows where there are few, a multiple of the rows worked on at a time.
Tiles tiles_of(const la_norm_shape& s, int elems, int arrays, int bytes, int stages) {
    Tiles t{};
    const int elem = elem_of(s.dtype), threads = row_threads(s.C, elems), at_once = block_for(threads) / threads;
    t.rows = s.rows;
    t.C = s.C;
    t.row = (uint32_t)s.C * elem;
    long long r = bytes / (long long)t.row, share = s.rows / (152 * 4);
    if (r > share) r = share;
    t.R = (int)(r / at_once * at_once);
    if (t.R < at_once) t.R = at_once;
    t.tiles = (s.rows + t.R - 1) / t.R;
    const long long fit = (long long)kMostSmem / ((long long)arrays * t.R * t.row);
    t.stages = (int)(fit < stages ? fit : stages);
    return t;
}
int resident(size_t smem, int most) {
    const long long per = (long long)kMostSmem / (long long)(smem + 1536);
    return (int)(per < 1 ? 1 : per > most ? most : per);
}
constexpr int kFwdTile = 8192, kBwdTile = 8192, kFwdStages = 3, kBwdStages = 2, kElementsPerSm = 5;
// Blocks of the gradient, i.e. its records of 3 C floats: the same whether or not there are a and dh.
int bwd_blocks(const la_norm_shape& s) {
    if (!bwd_streams(s)) {
        const int threads = row_threads(s.C, kBwdSingles), at_once = block_for(threads) / threads;
        const long long tiles = (s.rows + at_once - 1) / at_once, most = 152LL * (threads > 256 ? 1 : kElementsPerSm);
        return (int)(tiles < most ? tiles : most);
    }
    const int threads = row_threads(s.C, kBwdElems);
    const Tiles t = tiles_of(s, kBwdElems, 4, kBwdTile, kBwdStages);
    const long long most = 152LL * resident((size_t)4 * t.stages * t.R * t.row, threads > 256 ? 1 : 2);
    return (int)(t.tiles < most ? t.tiles : most);
}

// Calls go with (elements to a thread) / per and threads to a row of a size.
#define LA_ROW_SIZES(go, elems, per)                                   \
    switch (row_threads(s.C, elems)) {                                 \
        case 8: return go(elems / (per), 8);                           \
        case 16: return go(elems / (per), 16);                         \
        case 32: return go(elems / (per), 32);                         \
        case 64: return go(elems / (per), 64);                         \
        case 128: return go(elems / (per), 128);                       \
        case 256: return go(elems / (per), 256);                       \
        default:                                                       \
            if (s.C <= 512 * elems) return go(elems / (per), 512);     \
            if (s.C <= 512 * 16) return go(16 / (per), 512);           \
            return go(32 / (per), 512);                                \
    }

template <typename T>
cudaError_t resid_fwd_t(const ResidFwd& a, const la_norm_shape& s, bool rms, float eps, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const int threads = row_threads(s.C, vectors(s.C, sizeof(T)) ? kFwdElems : kFwdSingles), block = block_for(threads);
    if (!vectors(s.C, sizeof(T))) {
        const long long tiles = (s.rows + block / threads - 1) / (block / threads), most = 152LL * 16;
        const long long blocks = tiles < most ? tiles : most;
#define LA_GO(vpt, tpr)                                                                                                    \
    run("resid_fwd", resid_fwd_elements<T, vpt, tpr>, blocks, block, 0, st, (const T*)a.x, (const T*)a.a, (const T*)a.scale, \
        (const T*)a.w, (const T*)a.b, (T*)a.h, (T*)a.y, a.mean, a.rstd, s.rows, s.C, (int)rms, eps)
        LA_ROW_SIZES(LA_GO, kFwdSingles, 1)
#undef LA_GO
    }
    const Tiles t = tiles_of(s, kFwdElems, 2, kFwdTile, kFwdStages);
    const size_t smem = (size_t)2 * t.stages * t.R * t.row;
    const long long all = 152LL * resident(smem, 4), blocks = t.tiles < all ? t.tiles : all;
    auto go = [&](auto kern) {
        const cudaError_t e = allow_smem(kern, kMostSmem);
        if (e != cudaSuccess) return e;
        return run("resid_fwd", kern, blocks, block, smem, st, (const T*)a.x, (const T*)a.a, (const T*)a.scale, (const T*)a.w,
                   (const T*)a.b, (T*)a.h, (T*)a.y, a.mean, a.rstd, t, (int)rms, eps, device_error_word());
    };
#define LA_GO(vpt, tpr) go(resid_fwd_tiles<T, vpt, tpr>)
    LA_ROW_SIZES(LA_GO, kFwdElems, V)
#undef LA_GO
}

template <typename T>
cudaError_t resid_bwd_t(const ResidBwd& a, const la_norm_shape& s, bool rms, float* part, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const int threads = row_threads(s.C, bwd_streams(s) ? kBwdElems : kBwdSingles), block = block_for(threads), blocks = bwd_blocks(s);
    const size_t sums = block > threads ? (size_t)(block / threads) * s.C * 4 : 0;
    if (!bwd_streams(s)) {
#define LA_GO(vpt, tpr)                                                                                                       \
    run("resid_bwd", resid_bwd_elements<T, vpt, tpr>, blocks, block, sums, st, (const T*)a.h, (const T*)a.a, (const T*)a.scale, \
        (const T*)a.w, a.mean, a.rstd, (const T*)a.dy, (const T*)a.dh, (T*)a.dx, (T*)a.da, part, s.rows, s.C, (int)rms)
        LA_ROW_SIZES(LA_GO, kBwdSingles, 1)
#undef LA_GO
    }
    const int arrays = 2 + (a.dh ? 1 : 0) + (a.a ? 1 : 0);
    const Tiles t = tiles_of(s, kBwdElems, 4, kBwdTile, kBwdStages);  // of four arrays: the blocks do not depend on which are there
    size_t smem = (size_t)arrays * t.stages * t.R * t.row;
    const size_t one = (size_t)(block / threads) * s.C * 4;
    if (smem < one) smem = one;
    auto go = [&](auto kern) {
        const cudaError_t e = allow_smem(kern, kMostSmem);
        if (e != cudaSuccess) return e;
        return run("resid_bwd", kern, blocks, block, smem, st, (const T*)a.h, (const T*)a.a, (const T*)a.scale, (const T*)a.w,
                   a.mean, a.rstd, (const T*)a.dy, (const T*)a.dh, (T*)a.dx, (T*)a.da, part, t, (int)rms, device_error_word());
    };
#define LA_GO(vpt, tpr) go(resid_bwd_tiles<T, vpt, tpr>)
    LA_ROW_SIZES(LA_GO, kBwdElems, V)
#undef LA_GO
}

}  // namespace

size_t gated_bwd_bytes(const Gated& g) { return (size_t)gated_bwd_blocks(g) * g.D * 4; }

// The lanes of a row: 16 bytes each.
#define LA_HEADS(go)                                                                                  \
    switch (g.D) {                                                                                    \
        case 16: return g.dtype == LA_BF16 ? go(__nv_bfloat16, 2) : go(float, 4);                     \
        case 32: return g.dtype == LA_BF16 ? go(__nv_bfloat16, 4) : go(float, 8);                     \
        case 64: return g.dtype == LA_BF16 ? go(__nv_bfloat16, 8) : go(float, 16);                    \
        case 128: return g.dtype == LA_BF16 ? go(__nv_bfloat16, 16) : go(float, 32);                  \
    }                                                                                                 \
    return cudaErrorInvalidValue;
cudaError_t gated_fwd(const void* o, const void* gate, const void* w, void* y, const Gated& g, cudaStream_t st) {
#define LA_GO(T, L) gated_fwd_l<T, L>(o, gate, w, y, g, st)
    LA_HEADS(LA_GO)
#undef LA_GO
}
cudaError_t gated_bwd(const void* o, const void* gate, const void* w, const void* dy, void* dout, void* dgate, void* dw,
                      const Gated& g, char* ws, cudaStream_t st) {
    float* part = dw ? reinterpret_cast<float*>(ws) : nullptr;
#define LA_GO(T, L) gated_bwd_l<T, L>(o, gate, w, dy, dout, dgate, dw, g, part, st)
    LA_HEADS(LA_GO)
#undef LA_GO
}

size_t resid_bwd_bytes(const la_norm_shape& s) { return (size_t)bwd_blocks(s) * 3 * s.C * sizeof(float); }

cudaError_t resid_fwd(const ResidFwd& a, const la_norm_shape& s, bool rms, float eps, cudaStream_t st) {
    return s.dtype == LA_BF16 ? resid_fwd_t<__nv_bfloat16>(a, s, rms, eps, st) : resid_fwd_t<float>(a, s, rms, eps, st);
}

cudaError_t resid_bwd(const ResidBwd& in, const la_norm_shape& s, bool rms, char* ws, cudaStream_t st) {
    ResidBwd a = in;
    if (!a.dscale) a.a = nullptr;  // a is read for dscale only
    float* part = a.dw || a.db || a.dscale ? reinterpret_cast<float*>(ws) : nullptr;
    const cudaError_t e = s.dtype == LA_BF16 ? resid_bwd_t<__nv_bfloat16>(a, s, rms, part, st) : resid_bwd_t<float>(a, s, rms, part, st);
    if (e != cudaSuccess || !part) return e;
    const Outs outs{{a.dw, a.db, a.dscale}};
    const int K = a.dscale ? 3 : 2;  // without a the blocks leave the third sum out
    const long long grid = ((long long)K * s.C + 31) / 32;
    return s.dtype == LA_BF16 ? run("columns_join", columns_join_kernel<__nv_bfloat16>, grid, 1024, 0, st, (const float*)part, outs,
                                    bwd_blocks(s), s.C, K, 3 * s.C)
                              : run("columns_join", columns_join_kernel<float>, grid, 1024, 0, st, (const float*)part, outs,
                                    bwd_blocks(s), s.C, K, 3 * s.C);
}

}  // namespace bn
}  // namespace la
