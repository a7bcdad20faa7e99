// tc_path.h -- bf16 tensor-core (tcgen05 / TMEM / TMA) path, sm_100a.
#pragma once
#include <cuda.h>

#include "internal.h"

namespace gla {
namespace tc {
// 4-D bf16 tensor map: dims (innermost first), the byte strides of the outer three, box
// (b0, b1, 1, 1), 128-byte swizzle.
bool map4_bf16(CUtensorMap *m, const void *base, const uint64_t *dims, const uint64_t *strides, uint32_t b0, uint32_t b1);
}  // namespace tc
int tc_check(const Problem &p);
int selftest_timeout(unsigned *status, unsigned limit_us, cudaStream_t st);
size_t tc_workspace(const Problem &p, bool bwd);
int tc_fwd(const Problem &p, const void *q, const void *k, const void *v, const float *la, const float *h0,
           void *o, float *hT, void *ws, cudaStream_t st);
// The layer epilogue fused into the forward's output store: y = LayerNorm(o) w + b
// times r sigmoid(r), written beside o (tc_fwd_epilogue).
struct TcEpilogue {
  const void *r;
  const float *w, *b;
  float eps;
  void *y;
};
// bf16, a tensor-core shape, d_v a multiple of 128 up to 512, the fused variant,
// no reuse of segment contributions
bool tc_epilogue_fusable(const Problem &p);
int tc_fwd_epilogue(const Problem &p, const void *q, const void *k, const void *v, const float *la, const float *h0,
                    void *o, float *hT, const TcEpilogue &epi, void *ws, cudaStream_t st);
int tc_bwd(const Problem &p, const void *q, const void *k, const void *v, const float *la, const float *h0,
           const void *dout, const float *dhT, void *dq, void *dk, void *dv, float *dla, float *dh0, void *ws,
           cudaStream_t st);
int tc_fwd_state(const Problem &p, const void *q, const void *k, const void *v, const float *la, const float *h0,
                 float *delta, float *gamma, void *ws, cudaStream_t st);
int tc_bwd_state(const Problem &p, const void *q, const void *k, const float *la, const void *dout,
                 const float *dhT, float *ddelta, float *gamma, void *ws, cudaStream_t st);
}  // namespace gla
