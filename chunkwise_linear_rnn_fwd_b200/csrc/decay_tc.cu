// decay_tc.cu -- the decay-attention walk on tcgen05 tensor cores (bf16 tensors).
//
// Per chunk of 128 tokens (m of them live; reverse walks take chunks and tokens backwards
// and carry S' = lambda R, see decay.cu), with X, Y, Z the chunk's tiles:
//     O  = (X Y^T (.) D) Z + diag(f) X S ,    S <- lambda^m S + Y^T (diag(w) Z) ,
// D[i][j] = lambda^(i-j) below the diagonal, f_i = lambda^(i+1), w_j = lambda^(m-1-j): a
// constant decay makes them functions of the distance alone, one table per head, and no
// factor exceeds one.
//
// One CTA per (64 columns of V, segment, sequence and head) and one CTA per SM, 16 warps:
//   warp 0     TMA loads of X, Y, Z into a ring of chunks
//   warp 1     issues the products: dS = Y^T Zw (M = channels), X S and P Z (M = tokens,
//              two accumulators: the row factor f meets the first only), X Y^T
//   warps 4-7  scores from TMEM, times D, to bf16 in TMEM as the A operand of P Z; later
//              O from TMEM through a staging tile to global memory
//   warps 8-.. one thread per state row (channel): S in fp32 registers, dS from TMEM added,
//              a bf16 copy to shared memory as the B operand of the next chunk's X S
//   the rest   w (.) Z as a sum of two bf16 tiles (see below)
// The chain from chunk to chunk is dS -> state -> X S, beside it scores -> P -> P Z; the
// loads run ahead by the ring's depth.
//
// Precision: P and the copy of S that X S reads are rounded to bf16 (2^-8 of each term, the
// output's own rounding is as large).  The carried state is returned in fp32 and lives on
// through every later chunk, so its update must not lose that: Y is exact, and w (.) Z is
// split into a bf16 value and the bf16 rounding of what is left, 2^-16 of each term, at the
// price of a second product.  lambda^m multiplies the state once a chunk, thousands of
// times in a long sequence: it is applied as a sum of two fp32 numbers.
//
// 64 columns per CTA and not 128: the state, X S and the staging tile shrink, which leaves
// shared memory for two chunks in flight (one at 256 channels), and a batch of few heads
// fills twice the SMs.  X Y^T is computed again by every 64 columns; X and Y come from L2.
#include "decay.h"
#include "tc_common.cuh"
#include "tc_path.h"

namespace gla {
namespace {

constexpr int kC = 128;   // tokens of a chunk
constexpr int kBV = 64;   // columns of V per CTA
constexpr int kThreads = 512;
constexpr int kTmemCols = 512;
// TMEM columns: scores fp32, P bf16, the two output accumulators, dS per 128 channels
constexpr uint32_t kColSc = 0, kColP = 128, kColOa = 192, kColOb = 256, kColDs = 320;

// KB: 128-channel blocks of the contraction
template <int KB>
struct Smem {
  static constexpr int kStages = KB == 1 ? 2 : 1;
  static constexpr int kTile = kC * 128 * KB * 2;           // X or Y, SW128 blocks of 64 columns
  static constexpr int kZTile = kC * kBV * 2;
  static constexpr int x = 0, y = x + kStages * kTile, z = y + kStages * kTile, zh = z + kStages * kZTile,
                       zl = zh + kZTile, s = zl + kZTile, o = s + 128 * KB * kBV * 2, w = o + kZTile,
                       bar = w + 640, bytes = bar + 256;
  static_assert(bytes + 1024 <= kMaxDynSmem, "");
};

template <int KB, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
    k_decay_tc(const __grid_constant__ DecayWalk w, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ,
               const __grid_constant__ CUtensorMap tmO) {
  using L = Smem<KB>;
  constexpr int NS = L::kStages;
  constexpr int kStateWarps = 4 * KB;
  constexpr int kScale0 = KB == 1 ? 12 : 2, kScaleWarps = KB == 1 ? 4 : 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float *W = (float *)(smem + L::w);  // lambda^0 .. lambda^128
  uint64_t *bars = (uint64_t *)(smem + L::bar);
  uint64_t *xfull = bars, *xempty = xfull + NS, *yfull = xempty + NS, *yempty = yfull + NS, *zfull = yempty + NS,
           *zempty = zfull + NS, *scfull = zempty + NS, *pfull = scfull + 1, *ofull = pfull + 1, *oempty = ofull + 1,
           *dsfull = oempty + 1, *dsempty = dsfull + 1, *sfull = dsempty + 1, *qsdone = sfull + 1, *zready = qsdone + 1,
           *done = zready + 1;
  uint32_t *tslot = (uint32_t *)(done + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (w.V + kBV - 1) / kBV;
  const int vt = blockIdx.x % tiles, seg = blockIdx.y;
  const long bh = blockIdx.x / tiles;
  const int b = (int)(bh / w.H), h = (int)(bh % w.H), v0 = vt * kBV;
  const dev::DSeq sq = dev::decay_seq(w, b);
  const int n = (sq.len + kC - 1) / kC, nseg = max(1, (n + w.L - 1) / w.L);
  if (seg >= nseg || (!OUT && seg == nseg - 1)) return;  // the whole CTA
  int i0, i1;
  dev::decay_slots(w.s0, w.s1, w.alias, w.nseq, b, OUT ? w.status : nullptr, i0, i1);
  const double rate = dev::decay_rate(w.ld, h, w.status);
  const int c_begin = seg * w.L, nloc = max(0, min(n, c_begin + w.L) - c_begin);
  auto chunk_of = [&](int i) { return w.reverse ? n - 1 - (c_begin + i) : c_begin + i; };
  auto live_of = [&](int i) { return min(kC, sq.len - chunk_of(i) * kC); };
  const int ksteps = (w.K + 15) / 16, kblocks = (w.K + 63) / 64;

  if (tid == 0) {
    for (int i = 0; i < 6 * NS; ++i) dev::mbar_init(&xfull[i], 1);
    dev::mbar_init(scfull, 1);
    dev::mbar_init(pfull, 4);
    dev::mbar_init(ofull, 1);
    dev::mbar_init(oempty, 4);
    dev::mbar_init(dsfull, 1);
    dev::mbar_init(dsempty, kStateWarps);
    dev::mbar_init(sfull, kStateWarps);
    dev::mbar_init(qsdone, 1);
    dev::mbar_init(zready, kScaleWarps);
    dev::mbar_init(done, 1);
    dev::fence_mbar_init();
  }
  if (warp == 1) dev::tmem_alloc(tslot, kTmemCols);
  if (tid >= 128 && tid <= 128 + kC) W[tid - 128] = (float)dev::decay_pow(rate, tid - 128);
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tmem = *tslot;

  if (warp == 0) {
    // ============================ loads ============================
    if (lane == 0) {
      bool ok = true;
      int xi = 0, yi = 0, zi = 0;  // loads issued
      for (int i = 0; i < nloc && ok; ++i) {
        const int s = i % NS;
        const uint32_t ph = (uint32_t)((i / NS - 1) & 1);
        const int row = (int)(sq.row0 + (long)chunk_of(i) * kC);
        if (i >= NS) ok = dev::mbar_wait(&yempty[s], ph, w.status);
        if (!ok) break;
        dev::mbar_arrive_expect_tx(&yfull[s], (uint32_t)(kblocks * kC * 128));
        for (int cb = 0; cb < kblocks; ++cb)
          dev::tma_load_4d(smem + L::y + s * L::kTile + cb * kC * 128, &tmY, cb * 64, row, h, sq.b, &yfull[s]);
        ++yi;
        if (OUT) {
          if (i >= NS) ok = dev::mbar_wait(&xempty[s], ph, w.status);
          if (!ok) break;
          dev::mbar_arrive_expect_tx(&xfull[s], (uint32_t)(kblocks * kC * 128));
          for (int cb = 0; cb < kblocks; ++cb)
            dev::tma_load_4d(smem + L::x + s * L::kTile + cb * kC * 128, &tmX, cb * 64, row, h, sq.b, &xfull[s]);
          ++xi;
        }
        if (i >= NS) ok = dev::mbar_wait(&zempty[s], ph, w.status);
        if (!ok) break;
        dev::mbar_arrive_expect_tx(&zfull[s], (uint32_t)L::kZTile);
        dev::tma_load_4d(smem + L::z + s * L::kZTile, &tmZ, v0, row, h, sq.b, &zfull[s]);
        ++zi;
      }
      // every load issued lands before the CTA ends, also where a wait ran out
      for (int j = max(0, yi - NS); j < yi; ++j) (void)dev::mbar_wait(&yfull[j % NS], (uint32_t)((j / NS) & 1), w.status);
      for (int j = max(0, xi - NS); j < xi; ++j) (void)dev::mbar_wait(&xfull[j % NS], (uint32_t)((j / NS) & 1), w.status);
      for (int j = max(0, zi - NS); j < zi; ++j) (void)dev::mbar_wait(&zfull[j % NS], (uint32_t)((j / NS) & 1), w.status);
    }
  } else if (warp == 1) {
    // ============================ products ============================
    if (lane == 0) {
      constexpr uint32_t id_sc = dev::idesc_bf16(kC, kC, false, false);   // X, Y: K-major
      constexpr uint32_t id_o = dev::idesc_bf16(kC, kBV, false, true);    // X or P (TMEM); S or Z: MN-major
      constexpr uint32_t id_ds = dev::idesc_bf16(128, kBV, true, true);   // Y, Zw: MN-major
      const uint32_t sS = dev::smem_u32(smem + L::s), sZh = dev::smem_u32(smem + L::zh), sZl = dev::smem_u32(smem + L::zl);
      bool ok = true;
      auto scores = [&](int i) {
        const int s = i % NS;
        const uint32_t ph = (uint32_t)((i / NS) & 1);
        ok = dev::mbar_wait(&xfull[s], ph, w.status) && dev::mbar_wait(&yfull[s], ph, w.status);
        if (!ok) return;
        dev::tc_fence_after();
        const uint32_t sX = dev::smem_u32(smem + L::x + s * L::kTile), sY = dev::smem_u32(smem + L::y + s * L::kTile);
        for (int kk = 0; kk < ksteps; ++kk)
          dev::umma_bf16(tmem + kColSc, dev::desc_kmajor(sX, kC, 0, kk * 16), dev::desc_kmajor(sY, kC, 0, kk * 16), id_sc,
                         kk > 0 ? 1u : 0u);
        dev::umma_commit(scfull);
      };
      if (OUT && nloc > 0) scores(0);
      for (int i = 0; i < nloc && ok; ++i) {
        const int s = i % NS;
        const uint32_t ph = (uint32_t)((i / NS) & 1), par = (uint32_t)(i & 1);
        const int tsteps = (live_of(i) + 15) / 16;  // 16-token steps that hold a live token
        const uint32_t sX = dev::smem_u32(smem + L::x + s * L::kTile), sY = dev::smem_u32(smem + L::y + s * L::kTile),
                       sZ = dev::smem_u32(smem + L::z + s * L::kZTile);
        ok = dev::mbar_wait(&yfull[s], ph, w.status) && dev::mbar_wait(&zfull[s], ph, w.status) &&
             dev::mbar_wait(zready, par, w.status);
        if (ok && i > 0) ok = dev::mbar_wait(dsempty, par ^ 1u, w.status);
        if (!ok) break;
        dev::tc_fence_after();
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          for (int kk = 0; kk < tsteps; ++kk) {
            const uint64_t dy = dev::desc_mnmajor(sY, kC, kk * 16, 128 * kb);
            dev::umma_bf16(tmem + kColDs + kb * kBV, dy, dev::desc_mnmajor(sZh, kC, kk * 16, 0), id_ds, kk > 0 ? 1u : 0u);
            dev::umma_bf16(tmem + kColDs + kb * kBV, dy, dev::desc_mnmajor(sZl, kC, kk * 16, 0), id_ds, 1u);
          }
        dev::umma_commit(dsfull);
        dev::umma_commit(&yempty[s]);
        if (OUT) {
          ok = dev::mbar_wait(sfull, par, w.status);
          if (ok && i > 0) ok = dev::mbar_wait(oempty, par ^ 1u, w.status);
          if (!ok) break;
          dev::tc_fence_after();
          for (int kk = 0; kk < ksteps; ++kk)
            dev::umma_bf16(tmem + kColOb, dev::desc_kmajor(sX, kC, 0, kk * 16), dev::desc_mnmajor(sS, 128 * KB, kk * 16, 0),
                           id_o, kk > 0 ? 1u : 0u);
          dev::umma_commit(qsdone);
          dev::umma_commit(&xempty[s]);
          ok = dev::mbar_wait(pfull, par, w.status);
          if (!ok) break;
          dev::tc_fence_after();
          for (int kk = 0; kk < tsteps; ++kk)
            dev::umma_bf16_ts(tmem + kColOa, tmem + kColP + kk * 8, dev::desc_mnmajor(sZ, kC, kk * 16, 0), id_o,
                              kk > 0 ? 1u : 0u);
          dev::umma_commit(ofull);
        }
        dev::umma_commit(&zempty[s]);
        if (OUT && i + 1 < nloc) scores(i + 1);
      }
      dev::umma_commit(done);  // all products have completed before TMEM is released
      (void)dev::mbar_wait(done, 0, w.status);
    }
  } else if (warp >= kScale0 && warp < kScale0 + kScaleWarps) {
    // ============================ w (.) Z ============================
    const int t0 = tid - 32 * kScale0;
    bool ok = true;
    for (int i = 0; i < nloc; ++i) {
      const int s = i % NS;
      const uint32_t ph = (uint32_t)((i / NS) & 1);
      const int m = live_of(i), m16 = (m + 15) & ~15;
      if (ok) ok = dev::mbar_wait(&zfull[s], ph, w.status);
      if (ok && m < m16) ok = dev::mbar_wait(&yfull[s], ph, w.status);
      if (ok && i > 0) ok = dev::mbar_wait(dsfull, (uint32_t)((i - 1) & 1), w.status);
      if (ok) {
        uint8_t *zt = smem + L::z + s * L::kZTile;
        // a row is eight 16-byte units; their place in the swizzled row does not matter here
#pragma unroll 4
        for (int e = t0; e < m16 * 8; e += 32 * kScaleWarps) {
          const int r = e >> 3;
          uint4 u = *reinterpret_cast<const uint4 *>(zt + e * 16), hi, lo;
          // rows behind the sequence hold anything: zero times it must not be NaN
          if (r >= m) {
            u = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(zt + e * 16) = u;
          }
          const float f = W[r < m ? (w.reverse ? r + 1 : m - 1 - r) : 0];
          const uint32_t a[4] = {u.x, u.y, u.z, u.w};
          uint32_t ah[4], al[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = __uint_as_float(a[j] << 16) * f, q = __uint_as_float(a[j] & 0xffff0000u) * f;
            ah[j] = dev::pack_bf16(p, q);
            al[j] = dev::pack_bf16(p - __uint_as_float(ah[j] << 16), q - __uint_as_float(ah[j] & 0xffff0000u));
          }
          hi = make_uint4(ah[0], ah[1], ah[2], ah[3]);
          lo = make_uint4(al[0], al[1], al[2], al[3]);
          *reinterpret_cast<uint4 *>(smem + L::zh + e * 16) = hi;
          *reinterpret_cast<uint4 *>(smem + L::zl + e * 16) = lo;
        }
        uint8_t *yt = smem + L::y + s * L::kTile;
        const int dead = (m16 - m) * 8;
        for (int e = t0; e < dead * kblocks; e += 32 * kScaleWarps)
          *reinterpret_cast<uint4 *>(yt + (e / dead) * kC * 128 + m * 128 + (e % dead) * 16) = make_uint4(0, 0, 0, 0);
      }
      dev::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(zready);
    }
  } else if (warp >= 4 && warp < 8) {
    // ============================ P and O ============================
    if (OUT) {
      const int q4 = warp & 3, t = 32 * q4 + lane;
      const uint32_t lane_base = tmem + ((uint32_t)(32 * q4) << 16);
      uint8_t *stage = smem + L::o;
      const long rows = w.packed ? w.T : (long)w.nseq * w.T;
      bool ok = true;
      for (int i = 0; i < nloc; ++i) {
        const uint32_t par = (uint32_t)(i & 1);
        const int m = live_of(i);
        const long row0 = sq.row0 + (long)chunk_of(i) * kC;
        if (ok) ok = dev::mbar_wait(scfull, par, w.status);
        dev::tc_fence_after();
        // 32 columns (tokens j) at a time; blocks on the far side of the diagonal are zero
#pragma unroll 1
        for (int jb = 0; jb < 4; ++jb) {
          uint32_t p[16];
          if (w.reverse ? jb < q4 : jb > q4) {
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = 0u;
          } else {
            float sc[32];
            dev::tmem_ld32(lane_base + kColSc + 32 * jb, sc);
            dev::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int j = 32 * jb + e, g = w.reverse ? j - t : t - j;
              sc[e] = g >= 0 && j < m ? sc[e] * W[g & 127] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = dev::pack_bf16(sc[2 * e], sc[2 * e + 1]);
          }
          dev::tmem_st16u(lane_base + kColP + 16 * jb, p);
        }
        dev::tmem_wait_st();
        dev::tc_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(pfull);

        if (ok) ok = dev::mbar_wait(ofull, par, w.status);
        dev::tc_fence_after();
        const float f = W[t < m ? (w.reverse ? m - 1 - t : t + 1) : 0];
        if (tid == 128) dev::tma_store_wait_read();  // the store of the chunk before has read the tile
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float a[32], c[32];
          dev::tmem_ld32(lane_base + kColOa + 32 * hf, a);
          dev::tmem_ld32(lane_base + kColOb + 32 * hf, c);
          dev::tmem_wait_ld();
          if (hf == 1) {
            dev::tc_fence_before();
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(oempty);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = fmaf(f, c[e], a[e]);
          if ((w.acc_in || w.acc_out) && t < m && ok) {
            const long row = w.packed ? row0 + t : (long)b * w.T + row0 + t;
            float *part = w.acc + ((long)h * rows + row) * w.V + v0 + 32 * hf;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if (v0 + 32 * hf + e < w.V) {
                float4 x = make_float4(a[e], a[e + 1], a[e + 2], a[e + 3]);
                if (w.acc_in) {
                  const float4 y = *reinterpret_cast<const float4 *>(part + e);
                  x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                  a[e] = x.x, a[e + 1] = x.y, a[e + 2] = x.z, a[e + 3] = x.w;
                }
                if (w.acc_out) *reinterpret_cast<float4 *>(part + e) = x;
              }
          }
          const uint32_t so = dev::smem_u32(stage) + (uint32_t)t * 128u;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            dev::st_shared_v4(so + (uint32_t)(((4 * hf + j) ^ (t & 7)) << 4), dev::pack_bf16(a[8 * j], a[8 * j + 1]),
                              dev::pack_bf16(a[8 * j + 2], a[8 * j + 3]), dev::pack_bf16(a[8 * j + 4], a[8 * j + 5]),
                              dev::pack_bf16(a[8 * j + 6], a[8 * j + 7]));
        }
        dev::fence_proxy_async_smem();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (ok && !w.acc_out) {
          if (m == kC) {
            if (tid == 128) {
              dev::tma_store_4d(&tmO, stage, v0, (int)row0, h, sq.b);
              dev::tma_store_commit();
            }
          } else {  // rows behind the sequence are not this one's to write
            __nv_bfloat16 *o = (__nv_bfloat16 *)w.o.p + sq.b * w.o.sb + h * w.o.sh + row0 * w.o.st + v0;
            for (int e = tid - 128; e < m * 8; e += 128) {
              const int r = e >> 3, j = e & 7;
              if (v0 + 8 * j < w.V)
                *reinterpret_cast<uint4 *>(o + r * w.o.st + 8 * j) =
                    *reinterpret_cast<const uint4 *>(stage + r * 128 + ((j ^ (r & 7)) << 4));
            }
          }
        }
      }
      if (tid == 128) dev::tma_store_wait_all();
    }
  } else if (warp >= 8 && warp < 8 + kStateWarps) {
    // ============================ state ============================
    const int q4 = warp & 3, kb = (warp - 8) >> 2, kr = 128 * kb + 32 * q4 + lane;  // this thread's channel
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q4) << 16);
    const long KV = (long)w.K * w.V;
    float *wsb = w.ws + bh * w.P * KV + (long)kr * w.V + v0;
    const bool kok = kr < w.K;
    const int nv = min(kBV, w.V - v0);  // a multiple of 8
    const bool pass = w.P > 1 && nseg > 1;
    float S[kBV];
#pragma unroll
    for (int e = 0; e < kBV; ++e) S[e] = 0.f;
    if (kok) {
      if (OUT && pass) {
        // entry 0: the start state (segment 0); entries 1 .. seg: states of the segments before
        const float far = (float)dev::decay_pow(rate, (long)w.L * kC);
        for (int j = seg == 0 ? 0 : 1; j <= seg; ++j) {
          const float *u = wsb + j * KV;
#pragma unroll
          for (int e = 0; e < kBV; e += 4)
            if (e < nv) {
              const float4 x = *reinterpret_cast<const float4 *>(u + e);
              S[e] = fmaf(S[e], far, x.x), S[e + 1] = fmaf(S[e + 1], far, x.y);
              S[e + 2] = fmaf(S[e + 2], far, x.z), S[e + 3] = fmaf(S[e + 3], far, x.w);
            }
        }
      } else if (seg == 0) {
        if (i0 >= 0) {
          const float *u = w.s0.p + i0 * w.s0.slot + h * w.s0.head + kr * w.s0.row + v0 * w.s0.col;
          if (w.s0.col == 1) {
#pragma unroll
            for (int e = 0; e < kBV; e += 4)
              if (e < nv) {
                const float4 x = *reinterpret_cast<const float4 *>(u + e);
                S[e] = x.x, S[e + 1] = x.y, S[e + 2] = x.z, S[e + 3] = x.w;
              }
          } else {
#pragma unroll
            for (int e = 0; e < kBV; ++e)
              if (e < nv) S[e] = u[e * w.s0.col];
          }
        }
        if (!OUT) {
#pragma unroll
          for (int e = 0; e < kBV; e += 4)
            if (e < nv) *reinterpret_cast<float4 *>(wsb + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
        }
      }
    }
    const uint32_t srow = dev::smem_u32(smem + L::s) + (uint32_t)kr * 128u;
    auto publish = [&]() {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dev::st_shared_v4(srow + (uint32_t)((j ^ (kr & 7)) << 4), dev::pack_bf16(S[8 * j], S[8 * j + 1]),
                          dev::pack_bf16(S[8 * j + 2], S[8 * j + 3]), dev::pack_bf16(S[8 * j + 4], S[8 * j + 5]),
                          dev::pack_bf16(S[8 * j + 6], S[8 * j + 7]));
      dev::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(sfull);
    };
    if (OUT && nloc > 0) publish();
    int m_of = 0;
    float dh = 1.f, dl = 0.f;  // lambda^m as a sum
    bool ok = true;
    for (int i = 0; i < nloc; ++i) {
      const int m = live_of(i);
      if (m != m_of) {
        const double d = dev::decay_pow(rate, m);
        dh = (float)d;
        dl = (float)(d - (double)dh);
        m_of = m;
      }
      if (ok) ok = dev::mbar_wait(dsfull, (uint32_t)(i & 1), w.status);
      dev::tc_fence_after();
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float d[32];
        dev::tmem_ld32(lane_base + kColDs + kb * kBV + 32 * hf, d);
        dev::tmem_wait_ld();
        if (hf == 1) {
          dev::tc_fence_before();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(dsempty);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) S[32 * hf + e] = fmaf(S[32 * hf + e], dh, fmaf(S[32 * hf + e], dl, d[e]));
      }
      if (OUT && i + 1 < nloc) {
        if (ok) ok = dev::mbar_wait(qsdone, (uint32_t)(i & 1), w.status);
        publish();
      }
    }
    const bool last = seg == nseg - 1;
    if (kok && ok) {
      if (!OUT) {
#pragma unroll
        for (int e = 0; e < kBV; e += 4)
          if (e < nv)
            *reinterpret_cast<float4 *>(wsb + (seg + 1) * KV + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
      } else if (last && i1 >= 0) {
        float *u = w.s1.p + i1 * w.s1.slot + h * w.s1.head + kr * w.s1.row + v0 * w.s1.col;
        if (w.s1.col == 1) {
#pragma unroll
          for (int e = 0; e < kBV; e += 4)
            if (e < nv) *reinterpret_cast<float4 *>(u + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < kBV; ++e)
            if (e < nv) u[e * w.s1.col] = S[e];
        }
      }
    }
  }
  dev::tc_fence_before();
  __syncthreads();
  if (warp == 1) dev::tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------- host

bool ok_view(const DView &v, const DecayWalk &w) {
  // TMA: 16-byte base and distances, none of them zero where the axis has more than one
  // element, and below 2^40 bytes
  const bool dense = !w.packed && w.nseq > 1;
  auto fits = [](long s, bool used) { return !used || (s > 0 && s % 8 == 0 && s < (1L << 38)); };
  return ((uintptr_t)v.p & 15u) == 0 && fits(v.st, w.T > 1) && fits(v.sh, w.H > 1) && fits(v.sb, dense);
}

bool make_map(CUtensorMap *m, const DView &v, const DecayWalk &w, int channels) {
  const bool dense = !w.packed && w.nseq > 1;
  auto step = [](long s, bool used) { return (uint64_t)(used ? 2 * s : 16); };
  const uint64_t dims[4] = {(uint64_t)channels, (uint64_t)w.T, (uint64_t)w.H, (uint64_t)(dense ? w.nseq : 1)};
  const uint64_t strides[3] = {step(v.st, w.T > 1), step(v.sh, w.H > 1), step(v.sb, dense)};
  return tc::map4_bf16(m, v.p, dims, strides, 64, kC);
}

template <int KB>
int launch(const DecayWalk &w, cudaStream_t st) {
  CUtensorMap mx, my, mz, mo;
  if (!make_map(&mx, w.x, w, w.K) || !make_map(&my, w.y, w, w.K) || !make_map(&mz, w.z, w, w.V) ||
      !make_map(&mo, w.o, w, w.V))
    return GLA_ERR_CUDA;
  const int smem = Smem<KB>::bytes + 1024;
  if (cudaFuncSetAttribute(k_decay_tc<KB, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(k_decay_tc<KB, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return GLA_ERR_CUDA;
  const unsigned gx = (unsigned)((long)w.nseq * w.H * ((w.V + kBV - 1) / kBV));
  if (w.P > 1)
    GLA_LAUNCH(K_DECAY_STATES, st, (k_decay_tc<KB, false><<<dim3(gx, w.P - 1), kThreads, smem, st>>>(w, mx, my, mz, mo)));
  GLA_LAUNCH(K_DECAY_WALK, st, (k_decay_tc<KB, true><<<dim3(gx, w.P), kThreads, smem, st>>>(w, mx, my, mz, mo)));
  return GLA_OK;
}

}  // namespace

int decay_chunk_tc() { return kC; }

bool decay_tc_takes(const DecayWalk &w, int dtype) {
  return dtype == GLA_DTYPE_BF16 && w.K % 8 == 0 && w.V % 8 == 0 && ok_view(w.x, w) && ok_view(w.y, w) &&
         ok_view(w.z, w) && ok_view(w.o, w);
}

int decay_walk_tc(const DecayWalk &w, cudaStream_t st) { return w.K <= 128 ? launch<1>(w, st) : launch<2>(w, st); }

}  // namespace gla
