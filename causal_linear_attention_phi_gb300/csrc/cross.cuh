// cross.cuh -- cross attention: shapes, the split of its work over blocks, and the host launchers of its kernels.
//
// Work is a flat list of chunks of rows, head after head; a head of keys has as many as its batch entry's length asks
// for.  Of `ctas` blocks as many work as there are chunks, each with one at least (a block without any would leave a gap
// in a head's records); block c of those takes the chunks [total c / ctas, total (c + 1) / ctas), so that every block has the same share
// whatever the lengths are, and writes one record for each head that it meets.  Walking on, a block comes to a new (block,
// head) pair whenever either number grows, so block + head numbers the records without gaps that overlap.
#pragma once

#include <float.h>

#include "la_internal.cuh"

namespace la {
namespace cross {

// Rows of B Hk heads: keys (B batch entries of Hk heads, M rows of which the first lens[b] count; all where lens is null),
// or the queries of the heads of keys (lens null).
struct Rows {
    const int* lens;
    int B, Hk, M;
    __host__ __device__ int heads() const { return B * Hk; }
#ifdef __CUDACC__
    __device__ int live(int b) const { return lens ? min(max(lens[b], 0), M) : M; }
    // chunks of a head of batch entry b: those with a live row, or those without
    __device__ int chunks(int b, int chunk, bool dead) const {
        const int n = (live(b) + chunk - 1) / chunk;
        return dead ? (M + chunk - 1) / chunk - n : n;
    }
#endif
};

#ifdef __CUDACC__
// Sum of the chunks of a head over the batch entries before b.  A whole warp.
__device__ __forceinline__ long long chunks_before(const Rows& r, int b, int chunk, bool dead) {
    if (!r.lens) return (long long)b * r.chunks(0, chunk, dead);
    long long s = 0;
    for (int x = threadIdx.x & 31; x < b; x += 32) s += r.chunks(x, chunk, dead);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// A block's share of the work: its first chunk and how many it has.
struct Span {
    int bh, i;  // head, chunk of the head (among the live, or the dead ones)
    int left;   // chunks from there on (fewer than 2^31: a tensor has fewer than 2^40 elements, a chunk at least 2^10)
};
__device__ __forceinline__ Span span_of(const Rows& r, int chunk, bool dead, int cta, int ctas) {  // a whole warp
    const long long total = chunks_before(r, r.B, chunk, dead) * r.Hk;
    if (total < ctas) ctas = (int)total;
    if (cta >= ctas) return Span{0, 0, 0};
    long long from = total * cta / ctas;
    Span s{0, 0, (int)(total * (cta + 1) / ctas - from)};
    int b = 0;
    if (!r.lens) {
        const long long n = (long long)r.chunks(0, chunk, dead) * r.Hk;
        b = (int)(from / n);
        from -= b * n;
    } else {
        const int lane = threadIdx.x & 31;
        for (int base = 0;; base += 32) {  // ends: from < total
            const long long n = base + lane < r.B ? (long long)r.chunks(base + lane, chunk, dead) * r.Hk : 0;
            long long upto = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            const unsigned here = __ballot_sync(0xffffffffu, upto > from);
            if (here) {
                const int l = __ffs(here) - 1;
                b = base + l;
                from -= __shfl_sync(0xffffffffu, upto - n, l);
                break;
            }
            from -= __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    const int n = r.chunks(b, chunk, dead);
    s.bh = b * r.Hk + (int)(from / n);
    s.i = (int)(from % n);
    return s;
}

// The walk over a share.  `live` rows of the head; the chunk's rows are [i chunk, ...) (of the live ones).
struct Walk {
    Rows r;
    int chunk, bh, i, nch, live, left;
    bool fresh;  // no chunk of this head has been taken before
    __device__ Walk(const Rows& rows, int chunk_, const Span& s)
        : r(rows), chunk(chunk_), bh(s.bh), i(s.i), nch(0), live(0), left(s.left), fresh(true) {
        if (left > 0) {
            live = r.live(bh / r.Hk);
            nch = (live + chunk - 1) / chunk;
        }
    }
    __device__ bool more() const { return left > 0; }
    __device__ bool last() const { return left == 1 || i + 1 == nch; }  // of its head, for this block
    __device__ int row0() const { return i * chunk; }
    __device__ int rows() const { return min(chunk, live - i * chunk); }
    __device__ void next() {
        fresh = false;
        if (--left == 0 || ++i < nch) return;
        i = 0;
        fresh = true;
        do {  // ends: another chunk is left, so a later head has one
            ++bh;
            if ((bh % r.Hk) == 0 || r.Hk == 1) {
                live = r.live(bh / r.Hk);
                nch = (live + chunk - 1) / chunk;
            }
        } while (nch == 0);
    }
};

// The blocks whose records make up head bh: [first, last] (none where first > last).  A whole warp.
struct Range {
    int first, last;
};
__device__ __forceinline__ Range records_of(const Rows& r, int chunk, int bh, int ctas) {
    const int b = bh / r.Hk;
    const long long n = r.chunks(b, chunk, false), total = chunks_before(r, r.B, chunk, false) * r.Hk;
    if (n == 0) return Range{1, 0};
    if (total < ctas) ctas = (int)total;
    const long long from = chunks_before(r, b, chunk, false) * r.Hk + (bh - b * r.Hk) * n;
    // the block of chunk f is the largest c with floor(total c / ctas) <= f
    return Range{(int)(((from + 1) * ctas - 1) / total), (int)(((from + n) * ctas - 1) / total)};
}

// phi_f and dphi_from_phi, but a NaN stays one (fminf and fmaxf take the other operand: phi would be 1).
__device__ __forceinline__ float min_nan(float x, float y) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float phi_of(float x) {
    float high;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(high) : "f"(x), "f"(0.f));
    return high + ex2_approx(min_nan(x, 0.f) * 1.4426950408889634f);
}
__device__ __forceinline__ float slope_of(float phi) { return min_nan(phi, 1.f); }

// A head without keys is one whose z is 0 in every entry: its queries get 0 whatever they hold (0 times a NaN or infinity is not 0).

// 1 / den, and 0 for a query that no key answers: whose normaliser is 0, or below the normal numbers (phi is 0 there too; the
// inverse would overflow, and one such query with it dk and dv of its head).
__device__ __forceinline__ float over(float den) { return fabsf(den) < FLT_MIN ? 0.f : 1.f / den; }
#endif

constexpr int kSms = 152;
inline size_t up(size_t x) { return (x + 255) / 256 * 256; }  // a workspace region's bytes
#define CR_TRY(x)                            \
    do {                                     \
        const cudaError_t e_ = (x);          \
        if (e_ != cudaSuccess) return e_;    \
    } while (0)

inline long long query_rows(const la_cross_shape& s) { return (long long)(s.H / s.Hk) * s.N; }
inline Rows key_rows(const la_cross_shape& s, const int* lens) { return Rows{lens, s.B, s.Hk, s.M}; }
inline Rows grouped_queries(const la_cross_shape& s) { return Rows{nullptr, s.B * s.Hk, 1, (int)query_rows(s)}; }

struct FwdArgs {
    const void *q, *k, *v;
    const int* lens;
    void* o;
    float *S, *z;  // null, or receive the state
};
struct BwdArgs {
    const void *q, *k, *v;
    const int* lens;
    const float *S, *z;  // null, or the state
    const void* dout;
    void *dq, *dk, *dv;
};

bool tc_ok(const la_cross_shape& s);  // the tensor-core kernels serve this shape
size_t simt_bytes(const la_cross_shape& s, int op);
size_t tc_bytes(const la_cross_shape& s, int op);
cudaError_t simt_fwd(const FwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st);
cudaError_t simt_bwd(const BwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st);
cudaError_t simt_apply(const void* q, const float* S, const float* z, void* o, const la_cross_shape& s, cudaStream_t st);
cudaError_t tc_fwd(const FwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st);
cudaError_t tc_bwd(const BwdArgs& a, const la_cross_shape& s, char* ws, cudaStream_t st);
cudaError_t tc_apply(const void* q, const float* S, const float* z, void* o, const la_cross_shape& s, char* ws,
                     cudaStream_t st);
// A few rows of queries to a state: each state is read once, into registers.
cudaError_t apply_few(const void* q, const float* S, const float* z, void* o, const la_cross_shape& s, cudaStream_t st);

}  // namespace cross
}  // namespace la
