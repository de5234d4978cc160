// block_norm.cuh -- host launchers of the norms around a block: the gated norm of heads, the residual sum with a norm.
#pragma once

#include "la_internal.cuh"

namespace la {
namespace bn {

constexpr int kMaxC = 16384;

struct Gated {
    long long positions;  // B N
    int N, H, D;
    int dtype, rms;
    float eps;
};
size_t gated_bwd_bytes(const Gated& g);
cudaError_t gated_fwd(const void* o, const void* gate, const void* w, void* y, const Gated& g, cudaStream_t st);
cudaError_t gated_bwd(const void* o, const void* gate, const void* w, const void* dy, void* dout, void* dgate, void* dw,
                      const Gated& g, char* ws, cudaStream_t st);

struct ResidFwd {
    const void *x, *a, *scale, *w, *b;  // scale, w, b may be null
    void *h, *y;
    float *mean, *rstd;  // may be null
};
struct ResidBwd {
    const void *h, *a, *scale, *w;  // a, scale, w may be null
    const float *mean, *rstd;       // mean null for the root mean square
    const void *dy, *dh;            // dh may be null
    void *dx, *da, *dscale, *dw, *db;  // da, dscale, dw, db may be null
};
size_t resid_bwd_bytes(const la_norm_shape& s);
cudaError_t resid_fwd(const ResidFwd& a, const la_norm_shape& s, bool rms, float eps, cudaStream_t st);
cudaError_t resid_bwd(const ResidBwd& a, const la_norm_shape& s, bool rms, char* ws, cudaStream_t st);

}  // namespace bn
}  // namespace la
