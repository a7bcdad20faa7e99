// decay.cu -- decay attention (heads that forget at a constant rate): the C entries, the
// chunked walk on CUDA cores and the recurrent step.
#include "decay.h"

#include "decay_plan.h"
#include "tc_common.cuh"

namespace gla {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// ============================================================================
// The walk on CUDA cores.  A chunk of C tokens, m of them live:
//     o_i = sum_{j<=i} lambda^{i-j} (x_i . y_j) z_j + lambda^{i+1} x_i S ,
//     S  <- lambda^m S + sum_j lambda^{m-1-j} y_j^T z_j ,
// all weights at most one.  A reverse walk takes the chunks and the tokens of a chunk
// backwards and carries S' = lambda R, so that a start state enters its first token
// undecayed and the final state is dL/dS_0 itself: j >= i, lambda^{m-1-i} x_i S',
// S' <- lambda^m S' + sum_j lambda^{j+1} y_j^T z_j.
//
// CTA = (64 columns of V, segment, sequence and head), 256 threads as 16 x 16; x, y, z,
// the scores and the state live in shared memory in fp32.  Every product is a register
// tile per thread (4 x 4 at C = 64) fed by 16-byte shared-memory reads: rows 16 apart per
// thread and a row stride of 4 mod 32 words keep those free of bank conflicts.  Bound by
// fp32 arithmetic and shared-memory reads, not by HBM.
// ============================================================================
constexpr int kThreads = 256;
constexpr int kBV = kDecayTileV;

template <int C, int K>
struct CcSmem {
  static constexpr int KS = K + 4;
  static constexpr int PS = C + 4;
  static constexpr int x = 0, y = x + C * KS, z = y + C * KS, s = z + C * kBV, p = s + K * kBV, w = p + C * PS;
  static constexpr int wl = w + C + 4, floats = wl + C + 4;
};

__device__ __forceinline__ float4 load_quad(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 load_quad(const __nv_bfloat16 *p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

// whether four values at a time can be loaded: data, distances and width are multiples of four
template <typename T>
__device__ __forceinline__ bool quads(const T *p, long st, int n) {
  return ((uintptr_t)p & (4 * sizeof(T) - 1)) == 0 && st % 4 == 0 && n % 4 == 0;
}

// Rows [0, m) of n values, st apart, into [C][stride] padded with zeros to C x WIDTH; four
// loads of a thread are in flight together.
template <typename T, int C, int WIDTH>
__device__ __forceinline__ void load_tile(float *dst, int stride, const T *src, long st, int m, int n, bool wide) {
  constexpr int kRow = WIDTH / 4, kAll = C * kRow, kUnroll = kAll / kThreads < 4 ? kAll / kThreads : 4;
  static_assert(kAll % (kThreads * kUnroll) == 0, "");
#pragma unroll 1
  for (int e0 = threadIdx.x; e0 < kAll; e0 += kThreads * kUnroll) {
    float4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int e = e0 + u * kThreads, r = e / kRow, c = 4 * (e % kRow);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < m && c < n) {
        const T *p = src + r * st + c;
        if (wide) {
          v[u] = load_quad(p);
        } else {
          v[u].x = to_f(p[0]);
          if (c + 1 < n) v[u].y = to_f(p[1]);
          if (c + 2 < n) v[u].z = to_f(p[2]);
          if (c + 3 < n) v[u].w = to_f(p[3]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int e = e0 + u * kThreads;
      *reinterpret_cast<float4 *>(dst + (e / kRow) * stride + 4 * (e % kRow)) = v[u];
    }
  }
}

template <typename T, int C, int K, bool OUT, bool REV>
__global__ void __launch_bounds__(kThreads) k_decay_cc(DecayWalk w) {
  using L = CcSmem<C, K>;
  extern __shared__ __align__(16) float sm[];
  float *X = sm + L::x, *Y = sm + L::y, *Z = sm + L::z, *S = sm + L::s, *Pm = sm + L::p, *W = sm + L::w, *Wl = sm + L::wl;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int tiles = (w.V + kBV - 1) / kBV;
  const int vt = blockIdx.x % tiles, seg = blockIdx.y;
  const long bh = blockIdx.x / tiles;
  const int b = (int)(bh / w.H), h = (int)(bh % w.H), v0 = vt * kBV;
  const dev::DSeq sq = dev::decay_seq(w, b);
  const int n = (sq.len + C - 1) / C, nseg = max(1, (n + w.L - 1) / w.L);
  if (seg >= nseg || (!OUT && seg == nseg - 1)) {
    if (!OUT && w.pre_join && blockIdx.x == 0 && blockIdx.y == 0) dev::pdl_wait();
    return;
  }
  if (OUT && w.wait_first) dev::pdl_wait();
  if (!OUT || w.lead) dev::pdl_launch_dependents();
  int i0, i1;
  dev::decay_slots(w.s0, w.s1, w.alias, w.nseq, b, OUT ? w.status : nullptr, i0, i1);
  const double rate = dev::decay_rate(__ldg(w.ld + h), w.status);
  // lambda^i as W + Wl, W alone where it is not multiplied on
  for (int i = tid; i <= C; i += kThreads) {
    const double d = dev::decay_pow(rate, i);
    W[i] = (float)d;
    Wl[i] = (float)(d - (double)(float)d);
  }

  // ---- start state: thread (ty, tx) owns rows 4 ty + 64 i + e, columns 4 tx .. +3
  const long KV = (long)w.K * w.V;
  float *wsb = w.ws + bh * w.P * KV;
  const bool pass = w.P > 1 && nseg > 1;  // states come from and go to ws
  // lambda^(tokens of a segment) as a sum, like lambda^m below
  const double across = dev::decay_pow(rate, (long)w.L * C);
  const float far = (float)across, rest = (float)(across - (double)far);
  if (OUT && pass && !w.settled) dev::pdl_wait();
#pragma unroll 1
  for (int i = 0; i < K / 64 + (K % 64 ? 1 : 0); ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = 4 * ty + 64 * i + e;
      if (k >= K) continue;
      float4 v4;
      float *v = &v4.x;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int vc = v0 + 4 * tx + c;
        float a = 0.f;
        if (k < w.K && vc < w.V) {
          if (OUT && pass) {
            // entry 0: the start state (segment 0); entries 1 .. seg: states of the segments before
            const float *u = wsb + (long)k * w.V + vc;
            if (seg == 0) {
              a = u[0];
            } else {
              for (int j = 1; j <= seg; ++j) a = fmaf(a, far, fmaf(a, rest, u[j * KV]));
            }
          } else if (seg == 0 && i0 >= 0) {
            a = w.s0.p[i0 * w.s0.slot + h * w.s0.head + k * w.s0.row + vc * w.s0.col];
            if (!OUT) wsb[(long)k * w.V + vc] = a;
          } else if (!OUT && seg == 0) {
            wsb[(long)k * w.V + vc] = 0.f;
          }
        }
        v[c] = a;
      }
      *reinterpret_cast<float4 *>(S + k * kBV + 4 * tx) = v4;
    }

  const T *x = (const T *)w.x.p + sq.b * w.x.sb + h * w.x.sh + sq.row0 * w.x.st;
  const T *y = (const T *)w.y.p + sq.b * w.y.sb + h * w.y.sh + sq.row0 * w.y.st;
  const T *z = (const T *)w.z.p + sq.b * w.z.sb + h * w.z.sh + sq.row0 * w.z.st + v0;
  const int nv = min(kBV, w.V - v0);
  const bool wx = OUT && quads(x, w.x.st, w.K), wy = quads(y, w.y.st, w.K), wz = quads(z, w.z.st, nv);
  const long rows = w.packed ? w.T : (long)w.nseq * w.T;
  const int i_end = min(n, (seg + 1) * w.L);
  for (int i = seg * w.L; i < i_end; ++i) {
    const int c = REV ? n - 1 - i : i;
    const long t0 = (long)c * C;
    const int m = (int)min((long)C, sq.len - t0);
    __syncthreads();
    if (OUT) load_tile<T, C, K>(X, L::KS, x + t0 * w.x.st, w.x.st, m, w.K, wx);
    load_tile<T, C, K>(Y, L::KS, y + t0 * w.y.st, w.y.st, m, w.K, wy);
    load_tile<T, C, kBV>(Z, kBV, z + t0 * w.z.st, w.z.st, m, nv, wz);
    __syncthreads();
    constexpr int R = C / 16;
    if (OUT) {
      float s[R][R];
#pragma unroll
      for (int a = 0; a < R; ++a)
#pragma unroll
        for (int d = 0; d < R; ++d) s[a][d] = 0.f;
#pragma unroll 2
      for (int k = 0; k < K; k += 4) {
        float4 xv[R], yv[R];
#pragma unroll
        for (int a = 0; a < R; ++a) xv[a] = *reinterpret_cast<const float4 *>(X + (ty + 16 * a) * L::KS + k);
#pragma unroll
        for (int a = 0; a < R; ++a) yv[a] = *reinterpret_cast<const float4 *>(Y + (tx + 16 * a) * L::KS + k);
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
          for (int d = 0; d < R; ++d)
            if (REV ? d >= a : d <= a) {  // blocks of 16 x 16 on the diagonal's near side
              s[a][d] = fmaf(xv[a].x, yv[d].x, s[a][d]);
              s[a][d] = fmaf(xv[a].y, yv[d].y, s[a][d]);
              s[a][d] = fmaf(xv[a].z, yv[d].z, s[a][d]);
              s[a][d] = fmaf(xv[a].w, yv[d].w, s[a][d]);
            }
      }
#pragma unroll
      for (int a = 0; a < R; ++a)
#pragma unroll
        for (int d = 0; d < R; ++d) {
          const int t = ty + 16 * a, u = tx + 16 * d, g = REV ? u - t : t - u;
          Pm[t * L::PS + u] = g >= 0 ? s[a][d] * W[g] : 0.f;
        }
      __syncthreads();
      float4 in[R], ia[R];
#pragma unroll
      for (int a = 0; a < R; ++a) in[a] = ia[a] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < K; ++k) {
        const float4 sv = *reinterpret_cast<const float4 *>(S + k * kBV + 4 * tx);
#pragma unroll
        for (int a = 0; a < R; ++a) {
          const float q = X[(ty + 16 * a) * L::KS + k];
          in[a].x = fmaf(q, sv.x, in[a].x);
          in[a].y = fmaf(q, sv.y, in[a].y);
          in[a].z = fmaf(q, sv.z, in[a].z);
          in[a].w = fmaf(q, sv.w, in[a].w);
        }
      }
#pragma unroll
      for (int d = 0; d < R; ++d)
#pragma unroll 4
        for (int u = 16 * d; u < 16 * d + 16; ++u) {
          const float4 zv = *reinterpret_cast<const float4 *>(Z + u * kBV + 4 * tx);
#pragma unroll
          for (int a = 0; a < R; ++a)
            if (REV ? d >= a : d <= a) {
              const float q = Pm[(ty + 16 * a) * L::PS + u];
              ia[a].x = fmaf(q, zv.x, ia[a].x);
              ia[a].y = fmaf(q, zv.y, ia[a].y);
              ia[a].z = fmaf(q, zv.z, ia[a].z);
              ia[a].w = fmaf(q, zv.w, ia[a].w);
            }
        }
#pragma unroll
      for (int a = 0; a < R; ++a) {
        const int t = ty + 16 * a;
        if (t >= m) continue;
        const float f = W[REV ? m - 1 - t : t + 1];
        const float r[4] = {fmaf(f, in[a].x, ia[a].x), fmaf(f, in[a].y, ia[a].y), fmaf(f, in[a].z, ia[a].z),
                            fmaf(f, in[a].w, ia[a].w)};
        T *o = (T *)w.o.p + sq.b * w.o.sb + h * w.o.sh + (sq.row0 + t0 + t) * w.o.st + v0;
        const long row = w.packed ? sq.row0 + t0 + t : (long)b * w.T + t0 + t;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (4 * tx + e >= nv) continue;
          float val = r[e];
          float *part = w.acc + ((long)h * rows + row) * w.V + v0 + 4 * tx + e;
          if (w.acc_in) val += *part;
          if (w.acc_out) *part = val;
          else o[4 * tx + e] = from_f<T>(val);
        }
      }
      __syncthreads();  // S and Z are read
    }
    for (int e = tid; e < C * kBV; e += kThreads) {
      const int u = e / kBV;
      if (u < m) Z[e] *= W[REV ? u + 1 : m - 1 - u];
    }
    __syncthreads();
    // lambda^m as a sum: rounded to one fp32 number it is off the same way in every chunk, which
    // a slow head carries on (131072 tokens at log lambda = -1.08e-6: 6.1e-5 of the state, 2e-8 so)
    const float dh = W[m], dl = Wl[m];
#pragma unroll 1
    for (int i4 = 0; i4 < (K + 63) / 64; ++i4) {
      const int k0 = 4 * ty + 64 * i4;
      if (K % 64 != 0 && k0 >= K) continue;
      float4 d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = *reinterpret_cast<const float4 *>(S + (k0 + e) * kBV + 4 * tx);
      float4 f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int u = 0; u < C; ++u) {
        const float4 yv = *reinterpret_cast<const float4 *>(Y + u * L::KS + k0);
        const float4 zv = *reinterpret_cast<const float4 *>(Z + u * kBV + 4 * tx);
        const float q[4] = {yv.x, yv.y, yv.z, yv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e].x = fmaf(q[e], zv.x, f[e].x);
          f[e].y = fmaf(q[e], zv.y, f[e].y);
          f[e].z = fmaf(q[e], zv.z, f[e].z);
          f[e].w = fmaf(q[e], zv.w, f[e].w);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4 *>(S + (k0 + e) * kBV + 4 * tx) =
            make_float4(fmaf(d[e].x, dh, fmaf(d[e].x, dl, f[e].x)), fmaf(d[e].y, dh, fmaf(d[e].y, dl, f[e].y)),
                        fmaf(d[e].z, dh, fmaf(d[e].z, dl, f[e].z)), fmaf(d[e].w, dh, fmaf(d[e].w, dl, f[e].w)));
    }
  }

  // ---- the state after the segment: to ws, or to the pool after the sequence's last
  const bool last = seg == nseg - 1;
  if (!OUT || (last && i1 >= 0)) {
#pragma unroll 1
    for (int i = 0; i < (K + 63) / 64; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 4 * ty + 64 * i + e;
        if (k >= w.K || k >= K) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int vc = v0 + 4 * tx + c;
          if (vc >= w.V) continue;
          const float a = S[k * kBV + 4 * tx + c];
          if (!OUT) wsb[(seg + 1) * KV + (long)k * w.V + vc] = a;
          else w.s1.p[i1 * w.s1.slot + h * w.s1.head + k * w.s1.row + vc * w.s1.col] = a;
        }
      }
  }
  if ((OUT ? w.follows() : w.pre_join) && blockIdx.x == 0 && blockIdx.y == 0) dev::pdl_wait();
}

template <auto kernel>
int prepare(int smem) {  // a kernel's shared memory is set once per device
  static DeviceSlots slots;
  const int e = per_device(slots, [smem] {
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r != cudaSuccess) note_cuda_error(r);
    return r == cudaSuccess ? 1 : -1;
  });
  return e == 1 ? GLA_OK : GLA_ERR_CUDA;
}

template <typename T, int C, int K, bool REV>
int launch_cc(const DecayWalk &w, cudaStream_t st) {
  const int smem = CcSmem<C, K>::floats * 4;
  const unsigned gx = (unsigned)((long)w.nseq * w.H * ((w.V + kBV - 1) / kBV));
  if (w.P > 1 && (w.stage & 1)) {
    if (const int e = prepare<k_decay_cc<T, C, K, false, REV>>(smem)) return e;
    if (w.pre_join)
      GLA_LAUNCH(K_DECAY_STATES, st,
                 (void)launch_pdl(k_decay_cc<T, C, K, false, REV>, dim3(gx, w.P - 1), dim3(kThreads), smem, st, w));
    else
      GLA_LAUNCH(K_DECAY_STATES, st, (k_decay_cc<T, C, K, false, REV><<<dim3(gx, w.P - 1), kThreads, smem, st>>>(w)));
  }
  if (!(w.stage & 2)) return GLA_OK;
  if (const int e = prepare<k_decay_cc<T, C, K, true, REV>>(smem)) return e;
  if (w.follows())
    GLA_LAUNCH(K_DECAY_WALK, st,
               (void)launch_pdl(k_decay_cc<T, C, K, true, REV>, dim3(gx, w.P), dim3(kThreads), smem, st, w));
  else
    GLA_LAUNCH(K_DECAY_WALK, st, (k_decay_cc<T, C, K, true, REV><<<dim3(gx, w.P), kThreads, smem, st>>>(w)));
  return GLA_OK;
}

template <typename T, bool REV>
int walk_cc(const DecayWalk &w, cudaStream_t st) {
  if (w.K <= 64) return launch_cc<T, 64, 64, REV>(w, st);
  if (w.K <= 128) return launch_cc<T, 64, 128, REV>(w, st);
  return launch_cc<T, 32, 256, REV>(w, st);
}

// ============================================================================
// The recurrent step: one token per sequence.  Reads and rewrites the state once
// (2 * 4 * dk * dv bytes a head) and is bound by HBM on it, or by latency where the batch
// is small.  CTA = (4 CQ columns, sequence and head); a thread owns four columns and every
// RG-th row, kBatch of them loaded together, the first ones before anything else (a store
// between two loads of the state would hold the second back); the sums over the rows go
// through shared memory.
// ============================================================================
template <typename T, int CQ>  // CQ: quads of columns per CTA
__global__ void __launch_bounds__(256) k_decay_step(int H, int nseq, int K, int V, DView q, DView k, DView v, DView o,
                                                    const float *ld, DPool s, unsigned *status) {
  constexpr int RG = 256 / CQ, kBatch = 8;
  __shared__ float sq[256], sk[256];
  __shared__ float4 red[RG][CQ];
  const int tid = threadIdx.x, jq = tid % CQ, rg = tid / CQ;
  const int tiles = (V + 4 * CQ - 1) / (4 * CQ);
  const int vt = blockIdx.x % tiles;
  const long bh = blockIdx.x / tiles;
  const int b = (int)(bh / H), h = (int)(bh % H);
  int i0, i1;
  const DPool none{};
  dev::decay_slots(none, s, false, nseq, b, status, i0, i1);
  if (i1 < 0) return;
  const int col = vt * 4 * CQ + 4 * jq;
  float *S = s.p + i1 * s.slot + h * s.head + col;
  const bool quads = V % 4 == 0;  // the pool is 16-byte aligned
  const int nv = min(4, V - col);
  auto load = [&](int r) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < K) {
      const float *p = S + (long)r * V;
      if (quads) {
        if (nv > 0) x = *reinterpret_cast<const float4 *>(p);
      } else {
        if (nv > 0) x.x = p[0];
        if (nv > 1) x.y = p[1];
        if (nv > 2) x.z = p[2];
        if (nv > 3) x.w = p[3];
      }
    }
    return x;
  };
  float4 x[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) x[j] = load(rg + j * RG);
  // lambda as a sum: one fp32 number is up to 2^-25 off, which is 1 / 90 of what a head of
  // log lambda = -2.65e-6 forgets a token, and adds up over all of them
  const double lambda = dev::decay_pow(dev::decay_rate(__ldg(ld + h), status), 1);
  const float lh = (float)lambda, ll = (float)(lambda - (double)lh);
  if (tid < K) {
    sq[tid] = to_f(((const T *)q.p)[b * q.sb + h * q.sh + tid]);
    sk[tid] = to_f(((const T *)k.p)[b * k.sb + h * k.sh + tid]);
  }
  const T *vp = (const T *)v.p + b * v.sb + h * v.sh + col;
  float vv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e) vv[e] = e < nv ? to_f(vp[e]) : 0.f;
  __syncthreads();
  for (int r0 = rg;; r0 += RG * kBatch) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = r0 + j * RG;
      if (r >= K) continue;
      const float kr = sk[r], qr = sq[r];
      x[j].x = fmaf(lh, x[j].x, fmaf(ll, x[j].x, kr * vv[0]));
      x[j].y = fmaf(lh, x[j].y, fmaf(ll, x[j].y, kr * vv[1]));
      x[j].z = fmaf(lh, x[j].z, fmaf(ll, x[j].z, kr * vv[2]));
      x[j].w = fmaf(lh, x[j].w, fmaf(ll, x[j].w, kr * vv[3]));
      acc[0] = fmaf(qr, x[j].x, acc[0]);
      acc[1] = fmaf(qr, x[j].y, acc[1]);
      acc[2] = fmaf(qr, x[j].z, acc[2]);
      acc[3] = fmaf(qr, x[j].w, acc[3]);
      float *p = S + (long)r * V;
      if (quads) {
        if (nv > 0) *reinterpret_cast<float4 *>(p) = x[j];
      } else {
        if (nv > 0) p[0] = x[j].x;
        if (nv > 1) p[1] = x[j].y;
        if (nv > 2) p[2] = x[j].z;
        if (nv > 3) p[3] = x[j].w;
      }
    }
    if (r0 + RG * kBatch - rg >= K) break;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) x[j] = load(r0 + (kBatch + j) * RG);
  }
  red[rg][jq] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (tid < 4 * CQ) {
    const int c = vt * 4 * CQ + tid;
    if (c < V) {
      float sum = 0.f;
#pragma unroll 8
      for (int g = 0; g < RG; ++g) sum += (&red[g][tid / 4].x)[tid % 4];
      ((T *)o.p)[b * o.sb + h * o.sh + c] = from_f<T>(sum);
    }
  }
}

template <typename T, int CQ>
int launch_step(const gla_decay_desc &d, const DView &q, const DView &k, const DView &v, const DView &o, const float *ld,
                const DPool &s, cudaStream_t st) {
  const long grid = (long)d.B * d.H * ((d.dv + 4 * CQ - 1) / (4 * CQ));
  GLA_LAUNCH(K_DECAY_STEP, st,
             (k_decay_step<T, CQ><<<(unsigned)grid, 256, 0, st>>>(d.H, d.B, d.dk, d.dv, q, k, v, o, ld, s,
                                                                  (unsigned *)d.workspace)));
  return GLA_OK;
}

// 64 columns a CTA, or 16 where those would leave SMs idle
template <typename T>
int step(const gla_decay_desc &d, const DView &q, const DView &k, const DView &v, const DView &o, const float *ld,
         const DPool &s, cudaStream_t st) {
  if ((long)d.B * d.H * ((d.dv + 63) / 64) >= 2 * 148) return launch_step<T, 16>(d, q, k, v, o, ld, s, st);
  return launch_step<T, 4>(d, q, k, v, o, ld, s, st);
}

}  // namespace

int decay_walk_cc(const DecayWalk &w, int dtype, cudaStream_t st) {
  if (w.reverse) return dtype == GLA_DTYPE_BF16 ? walk_cc<__nv_bfloat16, true>(w, st) : walk_cc<float, true>(w, st);
  return dtype == GLA_DTYPE_BF16 ? walk_cc<__nv_bfloat16, false>(w, st) : walk_cc<float, false>(w, st);
}

namespace {

#define GLA_TRY(expr)            \
  do {                           \
    const int _r = (expr);       \
    if (_r != GLA_OK) return _r; \
  } while (0)

constexpr long kMaxHeads = 1 << 20;

int check_desc(const gla_decay_desc *d) {
  if (!d) return GLA_ERR_INVALID_ARG;
  if (d->B < 1 || d->H < 1 || d->T < 1 || d->dk < 1 || d->dv < 1 || d->segments < 0 || d->max_len < 0 ||
      d->max_len > d->T) return GLA_ERR_INVALID_ARG;
  if (d->dtype != GLA_DTYPE_BF16 && d->dtype != GLA_DTYPE_FP32) return GLA_ERR_INVALID_ARG;
  if (d->dk > 256 || d->dv > 4096 || (long)d->B * d->H > kMaxHeads || d->segments > kDecayMaxSegments)
    return GLA_ERR_UNSUPPORTED_SHAPE;
  return GLA_OK;
}

int check_view(const gla_view *v, int dtype, DView *out) {
  if (!v || !v->data || v->sb < 0 || v->sh < 0 || v->st < 0) return GLA_ERR_INVALID_ARG;
  if ((uintptr_t)v->data & (dtype == GLA_DTYPE_BF16 ? 1u : 3u)) return GLA_ERR_MISALIGNED;
  *out = DView{v->data, (long)v->sb, (long)v->sh, (long)v->st};
  return GLA_OK;
}

// an output: tokens, heads and sequences (one, if packed) that do not share their rows
int check_out(const gla_view *v, const gla_decay_desc *d, DView *out) {
  if (v && ((d->T > 1 && !v->st) || (d->H > 1 && !v->sh) || (d->B > 1 && !d->max_len && !v->sb))) return GLA_ERR_INVALID_ARG;
  return check_view(v, d->dtype, out);
}

int check_words(const void *p) { return (uintptr_t)p & 3u ? GLA_ERR_MISALIGNED : GLA_OK; }
int check_states(const float *p) { return ((uintptr_t)p & 15u) ? GLA_ERR_MISALIGNED : GLA_OK; }

DPool pool(const float *p, const int *idx, int slots, const gla_decay_desc *d, bool transposed) {
  const long KV = (long)d->dk * d->dv;
  return DPool{const_cast<float *>(p), idx, slots, d->H * KV, KV, transposed ? 1 : (long)d->dv,
               transposed ? (long)d->dv : 1};
}

size_t ws_bytes(const gla_decay_desc *d, bool bwd) {
  return kStatusBytes + decay_states_areas(d, bwd) * decay_states_bytes(d) + (bwd ? decay_acc_bytes(d) : 0);
}

int check_ws(const gla_decay_desc *d, bool bwd) {
  if (!d->workspace) return GLA_ERR_INVALID_ARG;
  if ((uintptr_t)d->workspace & 255u) return GLA_ERR_MISALIGNED;
  if (d->workspace_bytes < ws_bytes(d, bwd)) return GLA_ERR_WORKSPACE_TOO_SMALL;
  return GLA_OK;
}

// One walk by itself, its contraction over K channels in pieces of at most kDecayPiece.
int run_walk(DecayWalk w, const gla_decay_desc *d, cudaStream_t st) {
  const int K = w.K;
  const long es = d->dtype == GLA_DTYPE_BF16 ? 2 : 4;
  char *const x = (char *)w.x.p, *const y = (char *)w.y.p;
  float *const s0 = w.s0.p;
  const bool tc = decay_tc_takes(w, d->dtype);
  for (int k0 = 0; k0 < K; k0 += kDecayPiece) {
    const DecaySplit p = decay_split(d, tc, K, k0, w.V, decay_lines(d, w.V));
    w.K = p.K, w.P = p.P, w.L = p.L;
    w.x.p = x + k0 * es;
    w.y.p = y + k0 * es;
    if (s0) w.s0.p = s0 + k0 * w.s0.row;
    w.acc_in = k0 > 0;
    w.acc_out = k0 + kDecayPiece < K;
    GLA_TRY(tc ? decay_walk_tc(w, st) : decay_walk_cc(w, d->dtype, st));
  }
  return GLA_OK;
}

// Three walks that share nothing, each contraction in one piece: beside each other, split
// while together they leave SMs idle.  The pre-passes of those that are split come first.
// (4 heads of 8192 tokens of 128 x 256: 110 us; one after another, each split for itself,
// 199; whole beside each other 239.)
int run_together(DecayWalk *w, const gla_decay_desc *d, cudaStream_t st) {
  long lines = 0;
  for (int i = 0; i < 3; ++i) lines += decay_lines(d, w[i].V);
  bool tc[3], split = false;
  for (int i = 0; i < 3; ++i) {
    tc[i] = decay_tc_takes(w[i], d->dtype);
    const DecaySplit p = decay_split(d, tc[i], w[i].K, 0, w[i].V, lines);
    w[i].P = p.P, w[i].L = p.L;
    w[i].ws = (float *)((char *)w[i].ws + i * decay_states_bytes(d));
    if (w[i].P == 1) continue;
    w[i].stage = 1;
    w[i].pre_join = split;
    GLA_TRY(tc[i] ? decay_walk_tc(w[i], st) : decay_walk_cc(w[i], d->dtype, st));
    split = true;
  }
  for (int i = 0; i < 3; ++i) {
    w[i].stage = 2;
    w[i].wait_first = split && i == 0;
    w[i].settled = split && i > 0;
    w[i].join = i > 0;
    w[i].lead = i < 2;
    GLA_TRY(tc[i] ? decay_walk_tc(w[i], st) : decay_walk_cc(w[i], d->dtype, st));
  }
  return GLA_OK;
}

DecayWalk walk_base(const gla_decay_desc *d, const float *log_decay, const int *cu) {
  DecayWalk w{};
  w.nseq = d->B;
  w.H = d->H;
  w.T = d->T;
  w.packed = cu != nullptr;
  w.max_len = cu ? d->max_len : d->T;
  w.ld = log_decay;
  w.cu = cu;
  w.status = (unsigned *)d->workspace;
  w.ws = (float *)((char *)d->workspace + kStatusBytes);
  w.acc = (float *)((char *)w.ws + decay_states_bytes(d));
  w.stage = 3;
  return w;
}

int check_lengths(const gla_decay_desc *d, const int *cu) {
  if ((cu != nullptr) != (d->max_len > 0)) return GLA_ERR_INVALID_ARG;
  return check_words(cu);
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

size_t gla_decay_workspace_size(const gla_decay_desc *desc, int for_bwd) {
  if (check_desc(desc) != GLA_OK) return 0;
  return ws_bytes(desc, for_bwd != 0);
}

int gla_decay_fwd(const gla_decay_desc *desc, const gla_view *q, const gla_view *k, const gla_view *v,
                  const float *log_decay, const int *cu_seqlens, const float *h0, const int *h0_index,
                  const gla_view *o, float *h_final, const int *h_final_index, void *stream) {
  GLA_TRY(check_desc(desc));
  GLA_TRY(check_lengths(desc, cu_seqlens));
  if (!log_decay || (h0_index && !h0) || (h_final_index && !h_final)) return GLA_ERR_INVALID_ARG;
  if (h0 && (desc->slots0 < 1 || (!h0_index && desc->slots0 < desc->B))) return GLA_ERR_INVALID_ARG;
  if (h_final && (desc->slots1 < 1 || (!h_final_index && desc->slots1 < desc->B))) return GLA_ERR_INVALID_ARG;
  GLA_TRY(check_states(h0));
  GLA_TRY(check_states(h_final));
  for (const void *p : {(const void *)log_decay, (const void *)h0_index, (const void *)h_final_index}) GLA_TRY(check_words(p));
  GLA_TRY(check_ws(desc, false));
  DecayWalk w = walk_base(desc, log_decay, cu_seqlens);
  GLA_TRY(check_view(q, desc->dtype, &w.x));
  GLA_TRY(check_view(k, desc->dtype, &w.y));
  GLA_TRY(check_view(v, desc->dtype, &w.z));
  GLA_TRY(check_out(o, desc, &w.o));
  w.K = desc->dk;
  w.V = desc->dv;
  w.s0 = pool(h0, h0_index, desc->slots0, desc, false);
  w.s1 = pool(h_final, h_final_index, desc->slots1, desc, false);
  w.alias = h0 && h0 == h_final;
  return run_walk(w, desc, (cudaStream_t)stream);
}

int gla_decay_bwd(const gla_decay_desc *desc, const gla_view *q, const gla_view *k, const gla_view *v,
                  const float *log_decay, const int *cu_seqlens, const float *h0, const gla_view *do_,
                  const float *dh_final, const gla_view *dq, const gla_view *dk, const gla_view *dv, float *dh0,
                  void *stream) {
  GLA_TRY(check_desc(desc));
  GLA_TRY(check_lengths(desc, cu_seqlens));
  if (!log_decay) return GLA_ERR_INVALID_ARG;
  GLA_TRY(check_words(log_decay));
  for (const float *s : {h0, dh_final, (const float *)dh0}) GLA_TRY(check_states(s));
  GLA_TRY(check_ws(desc, true));
  DView vq, vk, vv, vdo, vdq, vdk, vdv;
  GLA_TRY(check_view(q, desc->dtype, &vq));
  GLA_TRY(check_view(k, desc->dtype, &vk));
  GLA_TRY(check_view(v, desc->dtype, &vv));
  GLA_TRY(check_view(do_, desc->dtype, &vdo));
  GLA_TRY(check_out(dq, desc, &vdq));
  GLA_TRY(check_out(dk, desc, &vdk));
  GLA_TRY(check_out(dv, desc, &vdv));
  cudaStream_t st = (cudaStream_t)stream;
  const int B = desc->B;
  DecayWalk w[3];
  for (DecayWalk &x : w) x = walk_base(desc, log_decay, cu_seqlens);
  w[0].K = desc->dv, w[0].V = desc->dk;  // dq = do S^T
  w[0].x = vdo, w[0].y = vv, w[0].z = vk, w[0].o = vdq;
  w[0].s0 = pool(h0, nullptr, B, desc, true);
  w[1].reverse = 1;  // dk = v R^T
  w[1].K = desc->dv, w[1].V = desc->dk;
  w[1].x = vv, w[1].y = vdo, w[1].z = vq, w[1].o = vdk;
  w[1].s0 = pool(dh_final, nullptr, B, desc, true);
  w[2].reverse = 1;  // dv = k R, dh0 = lambda R_1
  w[2].K = desc->dk, w[2].V = desc->dv;
  w[2].x = vk, w[2].y = vq, w[2].z = vdo, w[2].o = vdv;
  w[2].s0 = pool(dh_final, nullptr, B, desc, false);
  w[2].s1 = pool(dh0, nullptr, B, desc, false);
  if (desc->dv <= kDecayPiece) return run_together(w, desc, st);
  for (const DecayWalk &x : w) GLA_TRY(run_walk(x, desc, st));
  return GLA_OK;
}

int gla_decay_step(const gla_decay_desc *desc, const gla_view *q, const gla_view *k, const gla_view *v,
                   const float *log_decay, float *state, const int *index, const gla_view *o, void *stream) {
  if (!desc) return GLA_ERR_INVALID_ARG;
  gla_decay_desc d = *desc;
  d.T = 1;
  d.max_len = 0;
  d.segments = 0;
  GLA_TRY(check_desc(&d));
  if (!log_decay || !state || d.slots1 < 1 || (!index && d.slots1 < d.B)) return GLA_ERR_INVALID_ARG;
  GLA_TRY(check_states(state));
  GLA_TRY(check_words(log_decay));
  GLA_TRY(check_words(index));
  if ((uintptr_t)d.workspace & 3u) return GLA_ERR_MISALIGNED;
  DView vq, vk, vv, vo;
  GLA_TRY(check_view(q, d.dtype, &vq));
  GLA_TRY(check_view(k, d.dtype, &vk));
  GLA_TRY(check_view(v, d.dtype, &vv));
  GLA_TRY(check_out(o, &d, &vo));
  const DPool s = pool(state, index, d.slots1, &d, false);
  cudaStream_t st = (cudaStream_t)stream;
  return d.dtype == GLA_DTYPE_BF16 ? step<__nv_bfloat16>(d, vq, vk, vv, vo, log_decay, s, st)
                                   : step<float>(d, vq, vk, vv, vo, log_decay, s, st);
}

}  // extern "C"
