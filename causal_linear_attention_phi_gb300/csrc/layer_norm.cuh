// layer_norm.cuh -- host launchers of the layer norm kernels.
#pragma once

#include "la_internal.cuh"

namespace la {
namespace ln {

// Rows lie in shared memory, worked on by at most 512 threads; the gradient's keep dw and db of at most 32 columns each.
constexpr int kMaxC = 16384;

// Blocks of the gradient kernel, i.e. partial (dw, db) records of 2 C floats in the workspace.
int bwd_blocks(const la_norm_shape& s);
// w, b, mean, rstd may be null.
cudaError_t fwd(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, const la_norm_shape& s,
                float eps, cudaStream_t st);
// w may be null; dw and db may be null (both null: `part` is not used).
cudaError_t bwd(const void* x, const void* w, const float* mean, const float* rstd, const void* dy, void* dx, void* dw,
                void* db, float* part, const la_norm_shape& s, cudaStream_t st);

}  // namespace ln
}  // namespace la
