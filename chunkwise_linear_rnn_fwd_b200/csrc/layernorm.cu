// layernorm.cu -- layer norm over rows of d values, forward and backward (CUDA cores).
//
//     y = (x - mean) rstd w + b ,   rstd = 1 / sqrt(mean((x - mean)^2) + eps) ,
// and with x^ = (x - mean) rstd, g = dy w:
//     dx = rstd (g - mean(g) - x^ mean(g x^)) ,  dw = sum_rows dy x^ ,  db = sum_rows dy .
//
// Bound by HBM: the forward reads x and writes y, the backward reads x and dy and writes
// dx.  A row belongs to a group of G threads that hold it in registers, so it is read once:
// 16-byte loads where the data, the distance of rows and d allow, pairs of single values
// otherwise.  A CTA stays for many rows, its groups take them in turn, R at a time.
// Forward: up to 64 values a thread, a warp a row up to 2048 bf16 values, so that the sums
// over a row's threads are a small part (16384 rows of 2048: 30 us; 35 with 8 values a
// thread).  Backward: 8 values a thread, because each costs two more registers for its
// columns' sums over all rows, and what hides the latency here is the number of warps: 24 an
// SM at 80 registers.  (16384 rows of 1024: with 32 values a thread and 16 warps 57 us instead of
// 30, and rings of prefetched rows in shared memory did not make up for it; with 32 warps at
// 64 registers, which spill, 36.)  The sums over the threads of a row are formed for R rows
// together.  The backward leaves one partial sum of dw and db per CTA, which a second kernel
// adds in a fixed order.
#include <cuda_bf16.h>

#include "internal.h"
#include "tc_common.cuh"

namespace gla {
namespace {

// The arithmetic runs on pairs of fp32 values (f32x2: one instruction for two).
using dev::add2;
using dev::bf16pair;
using dev::f2;
using dev::fma2;
using dev::hsum;
using dev::mul2;
using dev::pk;
using dev::upk;

// VEC consecutive values of a tensor, 16 bytes or two values, as P pairs.  x may be y and dy
// may be dx (in place), so the loads are ordinary ones.
template <typename T, int VEC>
struct Pack;
template <>
struct Pack<float, 4> {
  static constexpr int P = 2;
  ulonglong2 a;
  __device__ __forceinline__ void load(const float *p) { a = *reinterpret_cast<const ulonglong2 *>(p); }
  __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<ulonglong2 *>(p) = a; }
  __device__ __forceinline__ f2 get(int i) const { return i ? a.y : a.x; }
  __device__ __forceinline__ void put(int i, f2 v) { (i ? a.y : a.x) = v; }
};
template <>
struct Pack<__nv_bfloat16, 8> {
  static constexpr int P = 4;
  uint32_t a[4];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    a[0] = u.x, a[1] = u.y, a[2] = u.z, a[3] = u.w;
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
    *reinterpret_cast<uint4 *>(p) = make_uint4(a[0], a[1], a[2], a[3]);
  }
  __device__ __forceinline__ f2 get(int i) const { return bf16pair(a[i]); }
  __device__ __forceinline__ void put(int i, f2 v) {
    float lo, hi;
    upk(v, lo, hi);
    a[i] = dev::pack_bf16(lo, hi);
  }
};
// two values loaded one by one; the second is absent (zero, not stored) behind a row's end
template <>
struct Pack<float, 2> {
  static constexpr int P = 1;
  f2 a;
  __device__ __forceinline__ void load(const float *p, bool both) { a = pk(p[0], both ? p[1] : 0.f); }
  __device__ __forceinline__ void store(float *p, bool both) const {
    float lo, hi;
    upk(a, lo, hi);
    p[0] = lo;
    if (both) p[1] = hi;
  }
  __device__ __forceinline__ f2 get(int) const { return a; }
  __device__ __forceinline__ void put(int, f2 v) { a = v; }
};
template <>
struct Pack<__nv_bfloat16, 2> {
  static constexpr int P = 1;
  uint32_t a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool both) {
    const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
    a = u[0] | (both ? (uint32_t)u[1] << 16 : 0u);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p, bool both) const {
    unsigned short *u = reinterpret_cast<unsigned short *>(p);
    u[0] = (unsigned short)(a & 0xffffu);
    if (both) u[1] = (unsigned short)(a >> 16);
  }
  __device__ __forceinline__ f2 get(int) const { return bf16pair(a); }
  __device__ __forceinline__ void put(int, f2 v) {
    float lo, hi;
    upk(v, lo, hi);
    a = dev::pack_bf16(lo, hi);
  }
};
template <typename T, int VEC>
__device__ __forceinline__ void load_pack(Pack<T, VEC> &p, const T *x, int c, int d) {
  if constexpr (VEC == 2) p.load(x + c, c + 1 < d);
  else p.load(x + c);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(const Pack<T, VEC> &p, T *x, int c, int d) {
  if constexpr (VEC == 2) p.store(x + c, c + 1 < d);
  else p.store(x + c);
}
// P pairs of weights from column c on (`none` without weights, zero behind the end)
template <int VEC, int P>
__device__ __forceinline__ void weights_of(const float *p, float none, int c, int d, f2 *v) {
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = pk(none, none);
  if (!p || c >= d) return;
  if constexpr (VEC == 2) {
    v[0] = pk(__ldg(p + c), c + 1 < d ? __ldg(p + c + 1) : 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      const ulonglong2 u = __ldg(reinterpret_cast<const ulonglong2 *>(p + c + 2 * i));
      v[i] = u.x, v[i + 1] = u.y;
    }
  }
}

constexpr int kBwdCtas = 444;  // three on each of 148 SMs: the most partial sums of a backward

// Sums of V values (V a power of two up to 8) over a group of G threads, each thread getting
// all of them.  Within a warp the values halve while the lanes they are summed over double:
// V - 1 exchanges and one more per halving that is left, not five a value.  Lane l then holds
// value l mod V.  Then through red[group][G / 32][V]; a group's threads alone meet at its barrier.
template <int G, int V>
__device__ __forceinline__ void group_sums(float (&x)[V], float *red) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = V / 2; half >= 1; half /= 2) {
    const bool up = (lane & half) != 0;
#pragma unroll
    for (int j = 0; j < half; ++j) {
      const float send = up ? x[j] : x[j + half], keep = up ? x[j + half] : x[j];
      x[j] = keep + __shfl_xor_sync(0xffffffffu, send, half);
    }
  }
  float s = x[0];
#pragma unroll
  for (int o = V; o < 32; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    const int group = threadIdx.x / G, warp = (threadIdx.x % G) >> 5;
    float *mine = red + group * W * V;
    if (lane < V) mine[warp * V + lane] = s;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(G) : "memory");
    // lane l adds value l mod V of the warps l / V, l / V + 32 / V, .. and the lanes the rest
    s = 0.f;
#pragma unroll
    for (int i = 0; i < W * V; i += 32)
      if (i + lane < W * V) s += mine[i + lane];
#pragma unroll
    for (int o = V; o < 32 && o < W * V; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = __shfl_sync(0xffffffffu, s, j);
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

// Threads of a CTA, and CTAs that an SM holds: as many as leave a thread the registers for its
// values (64 when 1024 threads stay, 80 when 768 do).
template <int G, bool BWD>
constexpr int threads_of() {
  return BWD && G <= 256 ? 256 : 512;
}
template <int VEC, int N, int G, int R, bool BWD>
constexpr int ctas_per_sm() {
  return BWD ? (N * VEC > 8 ? 1 : G <= 256 ? 3 : 2) : (N * VEC * R <= 16 ? 2 : 1);
}

template <typename T, int VEC, int N, int G, int R>
__global__ void __launch_bounds__(threads_of<G, false>(), ctas_per_sm<VEC, N, G, R, false>()) k_ln_fwd(LnArgs a) {
  constexpr int kGroups = threads_of<G, false>() / G, P = Pack<T, VEC>::P;
  // two places in turn: a thread past the barrier of one sum cannot reach the writes of the
  // sum after the next before every thread of its group has passed the next one's barrier
  __shared__ float red[2][kGroups * R * (G / 32)];
  const int t = threadIdx.x % G, group = threadIdx.x / G;
  const float inv = 1.f / (float)a.d;
  const long step = (long)gridDim.x * kGroups * R;
  for (long row0 = ((long)group * gridDim.x + blockIdx.x) * R; row0 < a.rows; row0 += step) {
    Pack<T, VEC> p[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const T *x = (const T *)a.x + (row0 + r) * a.ldx;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = VEC * (t + G * i);
        if (c < a.d && row0 + r < a.rows) load_pack(p[r][i], x, c, a.d);
      }
    }
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f2 s = pk(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (VEC * (t + G * i) < a.d)
#pragma unroll
          for (int e = 0; e < P; ++e) s = add2(s, p[r][i].get(e));
      mean[r] = hsum(s);
    }
    group_sums<G, R>(mean, red[0]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] *= inv;
      const f2 nm = pk(-mean[r], -mean[r]);
      f2 s = pk(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = VEC * (t + G * i);
        if (c < a.d)
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const f2 v = add2(p[r][i].get(e), VEC == 2 && c + 1 >= a.d ? pk(-mean[r], 0.f) : nm);
            s = fma2(v, v, s);
          }
      }
      rstd[r] = hsum(s);
    }
    group_sums<G, R>(rstd, red[1]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rstd[r] = rsqrtf(rstd[r] * inv + a.eps);
      if (t == 0 && row0 + r < a.rows) {
        if (a.mean) a.mean[row0 + r] = mean[r];
        if (a.rstd) a.rstd[row0 + r] = rstd[r];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = VEC * (t + G * i);
      f2 w[P], b[P];
      weights_of<VEC, P>(a.w, 1.f, c, a.d, w);
      weights_of<VEC, P>(a.b, 0.f, c, a.d, b);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const f2 nm = pk(-mean[r], -mean[r]), rs = pk(rstd[r], rstd[r]);
#pragma unroll
        for (int e = 0; e < P; ++e) p[r][i].put(e, fma2(mul2(add2(p[r][i].get(e), nm), rs), w[e], b[e]));
        if (c < a.d && row0 + r < a.rows) store_pack(p[r][i], (T *)a.out + (row0 + r) * a.ldo, c, a.d);
      }
    }
  }
}

// The groups of a backward CTA, where it has more than one, add up their sums in shared memory.
template <int VEC, int N, int G>
__host__ __device__ constexpr bool sums_in_smem() {
  static_assert(G == threads_of<G, true>() || 2 * VEC * N * G * sizeof(float) <= 40 * 1024,
                "the sums of a CTA with several groups");
  return G < threads_of<G, true>();
}

// Thread t of a group carries its columns' sums of dy x^ and dy over all of its rows.
template <typename T, int VEC, int N, int G, int R>
__global__ void __launch_bounds__(threads_of<G, true>(), ctas_per_sm<VEC, N, G, R, true>()) k_ln_bwd(LnArgs a) {
  constexpr int kGroups = threads_of<G, true>() / G, P = Pack<T, VEC>::P;
  __shared__ float red[2][kGroups * 2 * R * (G / 32)];  // in turn, as in the forward: one barrier a round
  extern __shared__ float shared_sums[];                // [2][d] (sums_in_smem)
  const int t = threadIdx.x % G, group = threadIdx.x / G;
  const float inv = 1.f / (float)a.d;
  const f2 zero = pk(0.f, 0.f);
  if (a.part) dev::pdl_launch_dependents();
  const long step = (long)gridDim.x * kGroups * R;
  f2 dw[N * P], db[N * P];
#pragma unroll
  for (int i = 0; i < N * P; ++i) dw[i] = db[i] = zero;
  constexpr bool kKeep = N * VEC <= 8;  // the weights stay in registers
  f2 wk[kKeep ? N * P : P];
  if constexpr (kKeep)
#pragma unroll
    for (int i = 0; i < N; ++i) weights_of<VEC, P>(a.w, 1.f, VEC * (t + G * i), a.d, wk + i * P);
  int par = 0;
  for (long row0 = ((long)group * gridDim.x + blockIdx.x) * R; row0 < a.rows; row0 += step, par ^= 1) {
    Pack<T, VEC> px[R][N], pg[R][N];
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long row = row0 + r;
      mean[r] = rstd[r] = 0.f;
      if (row < a.rows) {
        const T *x = (const T *)a.x + row * a.ldx, *dy = (const T *)a.dy + row * a.lddy;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = VEC * (t + G * i);
          if (c < a.d) load_pack(px[r][i], x, c, a.d), load_pack(pg[r][i], dy, c, a.d);
        }
        mean[r] = __ldg(a.cmean + row);
        rstd[r] = __ldg(a.crstd + row);
      }
    }
    float s[2 * R];  // sums of g and of g x^ (an absent value's dy and weight are zero)
    f2 s1[R], s2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s1[r] = s2[r] = zero;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = VEC * (t + G * i);
      f2 *w = wk + (kKeep ? i * P : 0);
      if constexpr (!kKeep) weights_of<VEC, P>(a.w, 1.f, c, a.d, w);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (c < a.d && row0 + r < a.rows) {
          const f2 nm = pk(-mean[r], -mean[r]), rs = pk(rstd[r], rstd[r]);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const f2 h = mul2(add2(px[r][i].get(e), nm), rs), dy = pg[r][i].get(e), g = mul2(dy, w[e]);
            dw[i * P + e] = fma2(dy, h, dw[i * P + e]);
            db[i * P + e] = add2(db[i * P + e], dy);
            s1[r] = add2(s1[r], g);
            s2[r] = fma2(g, h, s2[r]);
          }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) s[2 * r] = hsum(s1[r]), s[2 * r + 1] = hsum(s2[r]);
    group_sums<G, 2 * R>(s, red[par]);
    // dx = rstd g - rstd mean(g) - x^ rstd mean(g x^), x^ = x rstd - mean rstd
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = VEC * (t + G * i);
      f2 *w = wk + (kKeep ? i * P : 0);
      if constexpr (!kKeep) weights_of<VEC, P>(a.w, 1.f, c, a.d, w);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (c < a.d && row0 + r < a.rows) {
          const float mx = -rstd[r] * rstd[r] * (s[2 * r + 1] * inv), m1 = -rstd[r] * (s[2 * r] * inv) - mean[r] * mx;
          const f2 rs = pk(rstd[r], rstd[r]), c1 = pk(m1, m1), cx = pk(mx, mx);
          Pack<T, VEC> out;
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const f2 g = mul2(pg[r][i].get(e), w[e]);
            out.put(e, fma2(g, rs, fma2(px[r][i].get(e), cx, c1)));
          }
          store_pack(out, (T *)a.out + (row0 + r) * a.ldo, c, a.d);
        }
    }
  }
  if (!a.part) return;
  float *part = a.part + (long)blockIdx.x * 2 * a.d, *sums = shared_sums;
  // the CTA's groups in order
#pragma unroll 1
  for (int g = 0; g < kGroups; ++g) {
    if (g == group) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) {
          float u[2], v[2];
          upk(dw[i * P + e], u[0], u[1]);
          upk(db[i * P + e], v[0], v[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int c = VEC * (t + G * i) + 2 * e + k;
            if (c < a.d) {
              if (g > 0) u[k] += sums[c], v[k] += sums[a.d + c];
              float *to = g == kGroups - 1 ? part : sums;
              to[c] = u[k], to[a.d + c] = v[k];
            }
          }
        }
    }
    if (kGroups > 1) __syncthreads();
  }
}

// dw, db from the partial sums: a CTA owns 32 of the 2 d columns, warp v adds the partials
// v, v + 32, .. of its lane's column, then the first warp adds the 32 sums in order.
__global__ void __launch_bounds__(1024) k_ln_reduce(int parts, int d, const float *part, float *dw,
                                                    float *db) {
  __shared__ float red[32][33];
  dev::pdl_wait();  // launched while the backward drains: its partial sums are complete from here on
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

template <typename T, int VEC, int N, int G, int R, bool BWD>
int launch(const LnArgs &a, float *dw, float *db, cudaStream_t st) {
  // rows go to the CTAs first, then to their groups
  const long rounds = (a.rows + R - 1) / R, most = 148 * ctas_per_sm<VEC, N, G, R, BWD>();
  const unsigned grid = (unsigned)(rounds < most ? rounds : most);
  if constexpr (BWD) {
    const size_t smem = sums_in_smem<VEC, N, G>() && a.part ? (size_t)2 * a.d * sizeof(float) : 0;
    GLA_LAUNCH(K_LN_BWD, st, (k_ln_bwd<T, VEC, N, G, R><<<grid, threads_of<G, true>(), smem, st>>>(a)));
    if (a.part)
      GLA_LAUNCH(K_LN_REDUCE, st,
                 (void)launch_pdl(k_ln_reduce, dim3((2 * a.d + 31) / 32), dim3(1024), 0, st, (int)grid, a.d,
                                  (const float *)a.part, dw, db));
  } else {
    GLA_LAUNCH(K_LN_FWD, st, (k_ln_fwd<T, VEC, N, G, R><<<grid, threads_of<G, false>(), 0, st>>>(a)));
  }
  return GLA_OK;
}

// R rows at a time once there are enough for every group on the GPU
template <typename T, int VEC, int N, int G, int R, bool BWD>
int rows_of(const LnArgs &a, float *dw, float *db, cudaStream_t st) {
  if constexpr (R > 1)
    if (a.rows <= 148L * ctas_per_sm<VEC, N, G, R, BWD>() * (threads_of<G, BWD>() / G) * R / 2)
      return launch<T, VEC, N, G, 1, BWD>(a, dw, db, st);
  return launch<T, VEC, N, G, R, BWD>(a, dw, db, st);
}

// N packs a thread: a warp a row while that suffices (more rows at a time where less does),
// then more threads a row, then more packs.
template <typename T, int VEC, bool BWD>
int run(const LnArgs &a, float *dw, float *db, cudaStream_t st) {
  constexpr int R = sizeof(T) == 2 ? 2 : 1;
  if constexpr (BWD || VEC == 2) {
    constexpr int N = 8 / VEC, W = 32 * VEC * N;
    if (a.d <= W) return rows_of<T, VEC, N, 32, R, BWD>(a, dw, db, st);
    if (a.d <= 2 * W) return rows_of<T, VEC, N, 64, R, BWD>(a, dw, db, st);
    if (a.d <= 4 * W) return rows_of<T, VEC, N, 128, R, BWD>(a, dw, db, st);
    if (a.d <= 8 * W) return rows_of<T, VEC, N, 256, R, BWD>(a, dw, db, st);
    if (a.d <= 16 * W) return rows_of<T, VEC, N, 512, R, BWD>(a, dw, db, st);
    if (a.d <= 32 * W) return rows_of<T, VEC, 2 * N, 512, 1, BWD>(a, dw, db, st);
    return rows_of<T, VEC, 4 * N, 512, 1, BWD>(a, dw, db, st);
  } else {
    constexpr int N = 8, W = 32 * VEC * N;
    if (a.d <= W / 4) return rows_of<T, VEC, 2, 32, 4, BWD>(a, dw, db, st);
    if (a.d <= W / 2) return rows_of<T, VEC, 4, 32, 4, BWD>(a, dw, db, st);
    if (a.d <= W) return rows_of<T, VEC, N, 32, VEC == 8 ? 2 : 1, BWD>(a, dw, db, st);
    if (a.d <= 2 * W) return rows_of<T, VEC, N, 64, 1, BWD>(a, dw, db, st);
    if (a.d <= 4 * W) return rows_of<T, VEC, N, 128, 1, BWD>(a, dw, db, st);
    if (a.d <= 8 * W) return rows_of<T, VEC, N, 256, 1, BWD>(a, dw, db, st);
    return rows_of<T, VEC, N, 512, 1, BWD>(a, dw, db, st);
  }
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
  return align_up((size_t)(rows < kBwdCtas ? rows : kBwdCtas) * 2 * d * sizeof(float), 256);
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
  if (dtype == GLA_DTYPE_BF16)
    return wide ? run<__nv_bfloat16, 8, false>(a, nullptr, nullptr, st) : run<__nv_bfloat16, 2, false>(a, nullptr, nullptr, st);
  return wide ? run<float, 4, false>(a, nullptr, nullptr, st) : run<float, 2, false>(a, nullptr, nullptr, st);
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
    return wide ? run<__nv_bfloat16, 8, true>(a, dw, db, st) : run<__nv_bfloat16, 2, true>(a, dw, db, st);
  return wide ? run<float, 4, true>(a, dw, db, st) : run<float, 2, true>(a, dw, db, st);
}

}  // extern "C"
