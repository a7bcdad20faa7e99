// layernorm.cu -- layer norm over rows of d values, forward and backward (CUDA cores).
//
//     y = (x - mean) rstd w + b ,   rstd = 1 / sqrt(mean((x - mean)^2) + eps) ,
// and with x^ = (x - mean) rstd, g = dy w:
//     dx = rstd (g - mean(g) - x^ mean(g x^)) ,  dw = sum_rows dy x^ ,  db = sum_rows dy .
//
// Bound by HBM: the forward reads x and writes y, the backward reads x and dy and writes
// dx.  A row stays in the registers of a group of G threads (a warp, or a whole CTA for
// wide rows), so it is read once: 16-byte loads where the data, the distance of rows and d
// allow, single values otherwise.  The backward keeps the sums over rows for its columns
// in registers while it strides over the rows and leaves one partial sum per CTA; a second
// kernel adds those in a fixed order.
#include <cuda_bf16.h>

#include "internal.h"

namespace gla {
namespace {

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// VEC consecutive values as fp32 (VEC elements of T are 16 bytes, or one element)
template <int VEC>
__device__ __forceinline__ void ldv(const float *p, float *v) {
  if constexpr (VEC == 1) {
    v[0] = __ldg(p);
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    if constexpr (VEC == 8) {
      const float4 c = __ldg(reinterpret_cast<const float4 *>(p) + 1);
      v[4] = c.x, v[5] = c.y, v[6] = c.z, v[7] = c.w;
    }
  }
}
// x may be y and dy may be dx (in place): these are not read through the read-only path
template <typename T, int VEC>
struct Pack;
template <>
struct Pack<float, 4> {
  float4 a;
  __device__ __forceinline__ void load(const float *p) { a = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void get(float *v) const { v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w; }
  __device__ __forceinline__ void put(const float *v) { a = make_float4(v[0], v[1], v[2], v[3]); }
  __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = a; }
};
template <>
struct Pack<__nv_bfloat16, 8> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float *v) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void put(const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = a; }
};
template <>
struct Pack<float, 1> {
  float a;
  __device__ __forceinline__ void load(const float *p) { a = *p; }
  __device__ __forceinline__ void get(float *v) const { v[0] = a; }
  __device__ __forceinline__ void put(const float *v) { a = v[0]; }
  __device__ __forceinline__ void store(float *p) const { *p = a; }
};
template <>
struct Pack<__nv_bfloat16, 1> {
  __nv_bfloat16 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *p; }
  __device__ __forceinline__ void get(float *v) const { v[0] = __bfloat162float(a); }
  __device__ __forceinline__ void put(const float *v) { a = __float2bfloat16_rn(v[0]); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *p = a; }
};

// Sum over a group of G threads (G <= 32: within a warp; else the whole CTA of G threads,
// through `red`; every use gets its own slot of red, so one barrier a sum is enough)
template <int G>
__device__ __forceinline__ float group_sum(float x, float *red) {
  x = warp_sum(x);
  if constexpr (G > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < G / 32; ++i) x += red[i];
  }
  return x;
}

struct LnArgs {
  long rows;
  int d;
  const void *x, *dy;
  long ldx, lddy, ldo;
  const float *w, *b;
  float eps;
  void *out;
  float *mean, *rstd;          // forward: written where given
  const float *cmean, *crstd;  // backward
  float *part;                 // [CTAs][2][d]
};

constexpr int kLnThreads = 256;

// G threads hold N packs of VEC values of a row each.
template <typename T, int VEC, int N, int G>
__global__ void __launch_bounds__(G < kLnThreads ? kLnThreads : G) k_ln_fwd(LnArgs a) {
  __shared__ float red[2][32];
  constexpr int kGroups = G < kLnThreads ? kLnThreads / G : 1;
  const int t = threadIdx.x % G;
  const long row = (long)blockIdx.x * kGroups + threadIdx.x / G;
  if (row >= a.rows) return;  // a whole warp, or the whole CTA
  const T *x = (const T *)a.x + row * a.ldx;
  T *y = (T *)a.out + row * a.ldo;
  Pack<T, VEC> p[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = VEC * (t + G * i);
    if (c < a.d) p[i].load(x + c);
  }
  const float inv = 1.f / (float)a.d;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float v[VEC];
    p[i].get(v);
    if (VEC * (t + G * i) < a.d)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += v[e];
  }
  const float mean = group_sum<G>(s, red[0]) * inv;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float v[VEC];
    p[i].get(v);
    if (VEC * (t + G * i) < a.d)
#pragma unroll
      for (int e = 0; e < VEC; ++e) q = fmaf(v[e] - mean, v[e] - mean, q);
  }
  const float rstd = rsqrtf(group_sum<G>(q, red[1]) * inv + a.eps);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = VEC * (t + G * i);
    if (c < a.d) {
      float v[VEC], w[VEC], b[VEC];
      p[i].get(v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = 1.f, b[e] = 0.f;
      if (a.w) ldv<VEC>(a.w + c, w);
      if (a.b) ldv<VEC>(a.b + c, b);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = fmaf((v[e] - mean) * rstd, w[e], b[e]);
      p[i].put(v);
      p[i].store(y + c);
    }
  }
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// A group of G threads (a warp, or the whole CTA for wide rows) takes R rows at a time;
// thread t of it owns the columns VEC (t + G i) .. in every row and carries their sums of
// dy x^ and dy.  The next rows' loads are issued before these are worked on.
template <typename T, int VEC, int N, int G, int R>
__global__ void __launch_bounds__(G < kLnThreads ? kLnThreads : G, G <= kLnThreads ? 2 : 1) k_ln_bwd(LnArgs a) {
  constexpr int kGroups = G < kLnThreads ? kLnThreads / G : 1;
  __shared__ float2 red[2][R][32];
  extern __shared__ float sums[];  // [groups][2][d], with more than one group
  const int t = threadIdx.x % G, warp = threadIdx.x >> 5, group = threadIdx.x / G;
  const float inv = 1.f / (float)a.d;
  const long step = (long)gridDim.x * kGroups * R;
  float dw[N * VEC], db[N * VEC];
#pragma unroll
  for (int i = 0; i < N * VEC; ++i) dw[i] = db[i] = 0.f;
  // wide rows (many values a thread) keep neither the weights nor the next rows
  constexpr bool kKeep = N * VEC <= 16;
  struct Rows {
    Pack<T, VEC> x[R][N], g[R][N];
    float mean[R], rstd[R];
  };
  auto load = [&](Rows &p, long row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long row = row0 + r;
      p.mean[r] = p.rstd[r] = 0.f;
      if (row < a.rows) {
        const T *x = (const T *)a.x + row * a.ldx, *dy = (const T *)a.dy + row * a.lddy;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = VEC * (t + G * i);
          if (c < a.d) p.x[r][i].load(x + c), p.g[r][i].load(dy + c);
        }
        p.mean[r] = __ldg(a.cmean + row);
        p.rstd[r] = __ldg(a.crstd + row);
      }
    }
  };
  float kept[kKeep ? N * VEC : 1];
  auto weights = [&](int i, float *w) {
    const int c = VEC * (t + G * i);
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = 1.f;
    if (c < a.d && a.w) ldv<VEC>(a.w + c, w);
  };
  if constexpr (kKeep)
#pragma unroll
    for (int i = 0; i < N; ++i) weights(i, kept + i * VEC);
  int par = 0;
  long row0 = ((long)blockIdx.x * kGroups + group) * R;
  Rows p;
  load(p, row0);
  // (G > 32: one group a CTA, so that every thread makes the same number of rounds)
  for (; row0 < a.rows; row0 += step, par ^= 1) {
    Rows next;
    if constexpr (kKeep) load(next, row0 + step);
    float s1[R], s2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s1[r] = s2[r] = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = VEC * (t + G * i);
      float w[VEC];
      if constexpr (!kKeep) weights(i, w);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (c < a.d && row0 + r < a.rows) {
          float xv[VEC], gv[VEC];
          p.x[r][i].get(xv);
          p.g[r][i].get(gv);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float h = (xv[e] - p.mean[r]) * p.rstd[r], g = gv[e] * (kKeep ? kept[kKeep ? i * VEC + e : 0] : w[e]);
            dw[i * VEC + e] = fmaf(gv[e], h, dw[i * VEC + e]);
            db[i * VEC + e] += gv[e];
            s1[r] += g;
            s2[r] = fmaf(g, h, s2[r]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s1[r] = warp_sum(s1[r]);
      s2[r] = warp_sum(s2[r]);
    }
    if constexpr (G > 32) {
      // two buffers in turn: a thread past the barrier of one round cannot reach the writes
      // of the round after the next before every thread has passed the next one's barrier
      if ((t & 31) == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) red[par][r][warp] = make_float2(s1[r], s2[r]);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s1[r] = s2[r] = 0.f;
#pragma unroll
        for (int i = 0; i < G / 32; ++i) s1[r] += red[par][r][i].x, s2[r] += red[par][r][i].y;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = VEC * (t + G * i);
      float w[VEC];
      if constexpr (!kKeep) weights(i, w);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (c < a.d && row0 + r < a.rows) {
          const float m1 = s1[r] * inv, m2 = s2[r] * inv;
          float xv[VEC], gv[VEC];
          p.x[r][i].get(xv);
          p.g[r][i].get(gv);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float h = (xv[e] - p.mean[r]) * p.rstd[r], g = gv[e] * (kKeep ? kept[kKeep ? i * VEC + e : 0] : w[e]);
            xv[e] = p.rstd[r] * (g - m1 - h * m2);
          }
          Pack<T, VEC> out;
          out.put(xv);
          out.store((T *)a.out + (row0 + r) * a.ldo + c);
        }
      }
    }
    if constexpr (kKeep) p = next;
    else load(p, row0 + step);
  }
  if (!a.part) return;
  float *part = a.part + (long)blockIdx.x * 2 * a.d;
  float *mine = kGroups > 1 ? sums + (long)group * 2 * a.d : part;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = VEC * (t + G * i) + e;
      if (c < a.d) mine[c] = dw[i * VEC + e], mine[a.d + c] = db[i * VEC + e];
    }
  if constexpr (kGroups > 1) {  // the CTA's groups in order
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.d; c += kLnThreads) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) s += sums[(long)g * 2 * a.d + c];
      part[c] = s;
    }
  }
}

// dw, db from the partial sums: a CTA owns 32 of the 2 d columns, warp v adds the partials
// v, v + 32, .. of its lane's column, then the first warp adds the 32 sums in order.
__global__ void __launch_bounds__(1024) k_ln_reduce(int parts, int d, const float *__restrict__ part, float *dw,
                                                    float *db) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long c = (long)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2L * d)
#pragma unroll 4
    for (int p = warp; p < parts; p += 32) s += part[(long)p * 2 * d + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2L * d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][lane];
    if (c < d) {
      if (dw) dw[c] = s;
    } else if (db) {
      db[c - d] = s;
    }
  }
}

constexpr int kBwdCtas = 296;  // partial sums of a backward at most: two CTAs on each of 148 SMs

long bwd_ctas(long rows) { return rows < kBwdCtas ? rows : kBwdCtas; }

template <typename T, int VEC, int N, int G>
int fwd_launch(const LnArgs &a, cudaStream_t st) {
  constexpr int kGroups = G < kLnThreads ? kLnThreads / G : 1;
  const long grid = (a.rows + kGroups - 1) / kGroups;
  GLA_LAUNCH(K_LN_FWD, st, (k_ln_fwd<T, VEC, N, G><<<(unsigned)grid, G < kLnThreads ? kLnThreads : G, 0, st>>>(a)));
  return GLA_OK;
}

template <typename T, int VEC, int N, int G, int R>
int bwd_launch(const LnArgs &a, float *dw, float *db, cudaStream_t st) {
  constexpr int kGroups = G < kLnThreads ? kLnThreads / G : 1;
  const long rounds = (a.rows + kGroups * R - 1) / (kGroups * R), most = bwd_ctas(a.rows);
  const long grid = rounds < most ? rounds : most;
  const size_t smem = kGroups > 1 && a.part ? (size_t)kGroups * 2 * a.d * sizeof(float) : 0;
  GLA_LAUNCH(K_LN_BWD, st, (k_ln_bwd<T, VEC, N, G, R><<<(unsigned)grid, G < kLnThreads ? kLnThreads : G, smem, st>>>(a)));
  if (a.part)
    GLA_LAUNCH(K_LN_REDUCE, st, (k_ln_reduce<<<(2 * a.d + 31) / 32, 1024, 0, st>>>((int)grid, a.d, a.part, dw, db)));
  return GLA_OK;
}

// Rows up to 2048 values wide (512 single ones) to a warp each, wider ones to a CTA.
template <typename T, int VEC>
int fwd_t(const LnArgs &a, cudaStream_t st) {
  const int n = (a.d + VEC - 1) / VEC;  // packs of a row
  constexpr int F = VEC == 1 ? 4 : VEC == 4 ? 2 : 1;  // packs per thread that make 8 values, or 4 single ones
  if (n <= 32 * F) return fwd_launch<T, VEC, F, 32>(a, st);
  if (n <= 32 * 4 * F) return fwd_launch<T, VEC, 4 * F, 32>(a, st);
  if constexpr (VEC > 1)
    if (n <= 32 * 8 * F) return fwd_launch<T, VEC, 8 * F, 32>(a, st);
  if (n <= 256 * 2 * F) return fwd_launch<T, VEC, 2 * F, 256>(a, st);
  return fwd_launch<T, VEC, 4 * F, VEC == 1 ? 1024 : 512>(a, st);
}
// Rows up to 512 values (128 single ones) to a warp each.  Four rows at a time keep 64 KB in
// flight on an SM; wide rows do with fewer.
template <typename T, int VEC>
int bwd_t(const LnArgs &a, float *dw, float *db, cudaStream_t st) {
  const int n = (a.d + VEC - 1) / VEC;
  constexpr int F = VEC == 1 ? 4 : VEC == 4 ? 2 : 1;
  if (n <= 32 * F) return bwd_launch<T, VEC, F, 32, 4>(a, dw, db, st);
  if constexpr (VEC > 1)
    if (n <= 64 * F) return bwd_launch<T, VEC, 2 * F, 32, 2>(a, dw, db, st);
  if (n <= 256 * F) return bwd_launch<T, VEC, F, 256, 4>(a, dw, db, st);
  if (n <= 512 * 2 * F) return bwd_launch<T, VEC, 2 * F, 512, 1>(a, dw, db, st);
  return bwd_launch<T, VEC, VEC == 1 ? 8 * F : 4 * F, 512, 1>(a, dw, db, st);
}

bool al16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

int check(int dtype, long long rows, int d) {
  if (dtype != GLA_DTYPE_BF16 && dtype != GLA_DTYPE_FP32) return GLA_ERR_INVALID_ARG;
  if (rows < 1 || d < 1) return GLA_ERR_INVALID_ARG;
  return d <= 16384 && rows < (1LL << 31) ? GLA_OK : GLA_ERR_UNSUPPORTED_SHAPE;
}
int check_rows(const void *p, long long ld, int dtype, int d) {
  if (!p || ld < d) return GLA_ERR_INVALID_ARG;
  return (uintptr_t)p & (dtype == GLA_DTYPE_BF16 ? 1u : 3u) ? GLA_ERR_MISALIGNED : GLA_OK;
}
int check_f32(const void *p) { return (uintptr_t)p & 3u ? GLA_ERR_MISALIGNED : GLA_OK; }

}  // namespace
}  // namespace gla

using namespace gla;

#define GLA_TRY(expr)            \
  do {                           \
    const int _r = (expr);       \
    if (_r != GLA_OK) return _r; \
  } while (0)

extern "C" {

size_t gla_layernorm_workspace_size(long long rows, int d) {
  if (check(GLA_DTYPE_FP32, rows, d) != GLA_OK) return 0;
  return align_up((size_t)bwd_ctas(rows) * 2 * d * sizeof(float), 256);
}

int gla_layernorm_fwd(int dtype, long long rows, int d, const void *x, long long ldx, const float *w, const float *b,
                      float eps, void *y, long long ldy, float *mean, float *rstd, void *stream) {
  GLA_TRY(check(dtype, rows, d));
  if (!(eps > 0.f && eps < 1.f)) return GLA_ERR_INVALID_ARG;
  GLA_TRY(check_rows(x, ldx, dtype, d));
  GLA_TRY(check_rows(y, ldy, dtype, d));
  for (const float *p : {w, b, (const float *)mean, (const float *)rstd}) GLA_TRY(check_f32(p));
  LnArgs a{};
  a.rows = (long)rows, a.d = d, a.x = x, a.ldx = (long)ldx, a.w = w, a.b = b, a.eps = eps;
  a.out = y, a.ldo = (long)ldy, a.mean = mean, a.rstd = rstd;
  const int vec = dtype == GLA_DTYPE_BF16 ? 8 : 4;
  const bool wide = d % vec == 0 && ldx % vec == 0 && ldy % vec == 0 && al16(x) && al16(y) && al16(w) && al16(b);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == GLA_DTYPE_BF16) return wide ? fwd_t<__nv_bfloat16, 8>(a, st) : fwd_t<__nv_bfloat16, 1>(a, st);
  return wide ? fwd_t<float, 4>(a, st) : fwd_t<float, 1>(a, st);
}

int gla_layernorm_bwd(int dtype, long long rows, int d, const void *x, long long ldx, const void *dy, long long lddy,
                      const float *mean, const float *rstd, const float *w, void *dx, long long lddx, float *dw,
                      float *db, void *workspace, size_t workspace_bytes, void *stream) {
  GLA_TRY(check(dtype, rows, d));
  GLA_TRY(check_rows(x, ldx, dtype, d));
  GLA_TRY(check_rows(dy, lddy, dtype, d));
  GLA_TRY(check_rows(dx, lddx, dtype, d));
  if (!mean || !rstd) return GLA_ERR_INVALID_ARG;
  for (const float *p : {w, mean, rstd, (const float *)dw, (const float *)db}) GLA_TRY(check_f32(p));
  LnArgs a{};
  if (dw || db) {
    if (!workspace) return GLA_ERR_INVALID_ARG;
    if ((uintptr_t)workspace & 255u) return GLA_ERR_MISALIGNED;
    if (workspace_bytes < gla_layernorm_workspace_size(rows, d)) return GLA_ERR_WORKSPACE_TOO_SMALL;
    a.part = (float *)workspace;
  }
  a.rows = (long)rows, a.d = d, a.x = x, a.ldx = (long)ldx, a.dy = dy, a.lddy = (long)lddy, a.w = w;
  a.cmean = mean, a.crstd = rstd, a.out = dx, a.ldo = (long)lddx;
  const int vec = dtype == GLA_DTYPE_BF16 ? 8 : 4;
  const bool wide = d % vec == 0 && ldx % vec == 0 && lddy % vec == 0 && lddx % vec == 0 && al16(x) && al16(dy) &&
                    al16(dx) && al16(w);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == GLA_DTYPE_BF16)
    return wide ? bwd_t<__nv_bfloat16, 8>(a, dw, db, st) : bwd_t<__nv_bfloat16, 1>(a, dw, db, st);
  return wide ? bwd_t<float, 4>(a, dw, db, st) : bwd_t<float, 1>(a, dw, db, st);
}

}  // extern "C"
