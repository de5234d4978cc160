// tc_gated_delta.cuh -- pieces shared by the tensor-core kernels of the gated delta rule: tile layouts and their
// descriptors, products issued from a converged warp, hi + lo splitting, the kernels' entry.
#pragma once

#include "gated_delta.cuh"
#include "shared_memory.cuh"
#include "tc_common.cuh"

namespace la {
namespace gd {
namespace tcgd {
using namespace sm100;
using tc::bf_hi;
using tc::bf_lo;

constexpr int kBlk = kC * 128;          // 64 rows x 64 bf16 columns, 128-byte swizzle
// The 64 x 64 matrices of a chunk, a hi and a lo tile each.  The write strengths are folded into them, so that no
// recurrence multiplies by beta: t beta and P beta (columns), and in the gradient's records t beta, P and beta t (rows).
constexpr int kMatF = 0, kMatP = 2 * kBlk, kMatR = 4 * kBlk;
constexpr int kMatsFwd = 4 * kBlk, kMatsBwd = 6 * kBlk;  // bytes of a chunk
constexpr int kFwdGates = 3 * kC * 4;  // gam, -gam, tail beta of the record
constexpr int kRevGates = 6 * kC * 4;  // and tail, beta, -beta gam

// Contiguous shared -> global copy, tracked by the issuing thread's bulk groups.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
// Shared-memory operands, as the low word of their descriptors (address and leading offset, in units of 16 bytes;
// the high word is the same for all): K-major (rows are M or N) and MN-major (rows are K) tiles, K step kk of 16.  A
// whole warp runs the issuing role and one elected lane issues, so that these words stay in uniform registers: with the
// role in a one-lane branch an instruction cost about 90 cycles to issue, more than it takes to run.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <int kLead = 16>
__device__ __forceinline__ uint32_t tile_desc(uint32_t addr) {
    return ((addr & 0x3FFFFu) >> 4) | ((uint32_t)(kLead >> 4) << 16);
}
__device__ __forceinline__ constexpr uint32_t step_k(int kk, int blk = kBlk) { return ((kk >> 2) * blk + (kk & 3) * 32) >> 4; }
__device__ __forceinline__ constexpr uint32_t step_mn(int kk) { return (kk * 2048) >> 4; }

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p;
}
// D[tmem] (+)= A[tmem] B[smem], and with both in shared memory, by the elected lane of a converged warp.
__device__ __forceinline__ void mma_ts1(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 bd;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 bd, {%2, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"(lead), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ss1(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 ad, {%1, %4};\n\tmov.b64 bd, {%2, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"(lead), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit1(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}
// Every kernel here starts so: wait for the previous grid, take the TMEM columns, and only then let the next
// grid's blocks be scheduled.  Blocks of several of these kernels fit on one SM: none holds columns while it
// waits for a grid, and none is still to take its columns when a block that waits for it can arrive.
__device__ __forceinline__ uint32_t enter(uint32_t* slot, uint32_t cols, int warp) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 1) {
        tmem_alloc(slot, cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    return *slot;
}
// Byte offset of 16-byte chunk c of row r in rows of 64 columns.
__device__ __forceinline__ int row_off(int r, int c) { return r * 128 + (((c & 7) ^ (r & 7)) << 4); }
// a, b -> packed bf16 hi and lo parts.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16x2(a, b);
    lo = pack_bf16x2(a - bf_lo(hi), b - bf_hi(hi));
}

constexpr int kWarps = 16;  // compute warps
constexpr int kThreads = 64 + 32 * kWarps;
constexpr int kHs = kWarps / 4;   // column groups: a thread owns one row of one group
constexpr int kTok = kC / kHs;    // positions of a thread

// 32 lanes x 8 consecutive 32-bit columns -> 8 registers per thread.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// 32 lanes x 8 consecutive 32-bit columns from 8 registers per thread.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
template <int N>
__device__ __forceinline__ void ld(uint32_t a, uint32_t (&r)[N]) {
    static_assert(N == 8 || N == 16 || N == 32, "columns");
    if constexpr (N == 8) tmem_ld8(a, r);
    if constexpr (N == 16) tmem_ld16(a, r);
    if constexpr (N == 32) tmem_ld32(a, r);
}
template <int N>
__device__ __forceinline__ void st(uint32_t a, const uint32_t (&r)[N]) {
    static_assert(N == 8 || N == 16 || N == 32, "columns");
    if constexpr (N == 8) tmem_st8(a, r);
    if constexpr (N == 16) tmem_st16(a, r);
    if constexpr (N == 32) tmem_st32(a, r);
}


// What is formed for a product goes to TMEM hi parts first, with a signal of their own: the products of the hi parts run
// while the lo parts are formed.  Values in pairs, as the packed arithmetic has them.
__device__ __forceinline__ float2 pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ uint32_t hi2(float2 v) { return pack_bf16x2(v.x, v.y); }
__device__ __forceinline__ uint32_t lo2(float2 v, uint32_t hi) {
    const float2 d = fma2v(make_float2(bf_lo(hi), bf_hi(hi)), make_float2(-1.f, -1.f), v);
    return pack_bf16x2(d.x, d.y);
}
template <int N>
__device__ __forceinline__ void put_hi(uint32_t a, const float2 (&v)[N], uint32_t (&hi)[N]) {
#pragma unroll
    for (int x = 0; x < N; ++x) hi[x] = hi2(v[x]);
    st(a, hi);
    tmem_st_wait();
}
template <int N>
__device__ __forceinline__ void put_lo(uint32_t a, const float2 (&v)[N], const uint32_t (&hi)[N]) {
    uint32_t lo[N];
#pragma unroll
    for (int x = 0; x < N; ++x) lo[x] = lo2(v[x], hi[x]);
    st(a, lo);
    tmem_st_wait();
}

// One column r of a tile of 64-column blocks (`blk` bytes apart), rows row0 (a multiple of 8) + x for constant x: the
// swizzle is an exclusive or of the row into bits 4-6 of the address, so an access is that and an immediate offset.
// Written for the shared address space: generic addressing took a dozen instructions an element, more than the rest of
// the phase.
__device__ __forceinline__ uint32_t col_addr(const void* tile, int r, int row0, int blk = kBlk) {
    return smem_u32(tile) + (r >> 6) * blk + row0 * 128 + ((r >> 3) & 7) * 16 + (r & 7) * 2;
}
__device__ __forceinline__ float col_get(uint32_t col, int x) {  // a bf16
    uint32_t v;
    asm volatile(
        "{\n\t.reg .b16 h, z;\n\tmov.b16 z, 0;\n\t"
        "ld.shared.b16 h, [%1];\n\tmov.b32 %0, {z, h};\n\t}"
        : "=r"(v)
        : "r"((col ^ ((x & 7) << 4)) + x * 128)
        : "memory");
    return __uint_as_float(v);
}
__device__ __forceinline__ void col_put(uint32_t col, int x, uint16_t v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"((col ^ ((x & 7) << 4)) + x * 128), "h"(v) : "memory");
}
// Two bf16 of rows x and x + 1.
__device__ __forceinline__ void col_put2(uint32_t col, int x, float a, float b) {
    const uint32_t w = pack_bf16x2(a, b);
    col_put(col, x, (uint16_t)w);
    col_put(col, x + 1, (uint16_t)(w >> 16));
}

#define GD_TRY(x)                         \
    do {                                  \
        const cudaError_t _e = (x);       \
        if (_e != cudaSuccess) return _e; \
    } while (0)

// t and P of every chunk (tc_gated_delta.cu).
template <int D>
cudaError_t prepare(const CUtensorMap& tq, const CUtensorMap& tk, const void* g, const void* beta, float* recs,
                    uint8_t* mats, const la_shape& s, int M, bool bwd, int* err, cudaStream_t st);
// The recurrence's modes.  kOut: outputs.  kGrad: the gradient's records instead, for each chunk the state entering it
// (s_tiles, S^T as [Dv rows x Dk] bf16 tiles of 64 columns) and X (x_tiles, lo then hi, X^T as [Dv rows x 64
// positions]).  kSum: only the segment's last state, from a zero state (segB) and, with no values, from the identity
// (segM): the state after a segment is segB + segM (the state before it).
enum Mode { kOut, kGrad, kSum };
struct StateArgs {
    const float* recs;
    const uint8_t* mats;
    int mat_bytes;     // kMatsFwd or kMatsBwd
    const float* S0;   // [BH][P] records of dk x dv: the states entering the segments; null: zero
    int dk, dv;
    float* S_out;      // kOut: [BH] records, the state after the last position, or null
    __nv_bfloat16* o;  // kOut: [BH][N][Dv]
    int N, Dk, Dv;     // true sizes
    uint8_t *x_tiles, *s_tiles;   // kGrad
    float *segB, *segM;           // kSum: [BH][P] records
    int M, P, cps;                // chunks, segments, chunks of a segment
};
// Joins the segments' sums: out[p + 1] = B[p] + M[p] out[p] from out[0] = first and, where out2 is given, in reverse
// out2[p - 1] = B2[p] + M[p]^T out2[p] from out2[P - 1] = first2 (first, first2: Dk x Dv records; null: zero).
template <int D>
cudaError_t join(const float* B, const float* Mx, const float* first, float* out, const float* B2, const float* first2,
                 float* out2, int BH, int P, int Dk, int Dv, int* err, cudaStream_t st);

}  // namespace tcgd
}  // namespace gd
}  // namespace la
