// shared_memory.cuh -- what kernels may take of an SM's shared memory, and contiguous copies into it.
#pragma once

#include "la_internal.cuh"
#include "sm100.cuh"

namespace la {

// Opts a kernel in to `most` bytes of dynamic shared memory: the most that any of its calls takes, not this call's.  The
// limit belongs to the kernel and all host threads share it; set to a call's own size, a smaller call of another thread
// could lower it between this thread's setting and its launch, which then fails.
constexpr int kMaxHead = 128;  // the largest head size
template <typename K>
cudaError_t allow_smem(K kern, size_t most) {
    return cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

namespace sm100 {

// Contiguous global -> shared copy (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}
// After a wait that ran out: for copies that the calling thread has issued to `stages` buffers in turn (the i-th completes
// phase i / stages of barrier i % stages), waits once more, with the same limit, for those that may be in flight.  No block
// leaves copies behind, which would land in the shared memory of the next one.
inline __device__ __noinline__ void mbar_drain(uint64_t* bar, int stages, long long issued, int* err, int code) {
    for (long long i = issued > stages ? issued - stages : 0; i < issued; ++i)
        mbar_wait(bar + i % stages, (int)(i / stages) & 1, err, code);
}

}  // namespace sm100
}  // namespace la
