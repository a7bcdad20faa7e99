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
//   warps 0-3  one issues the TMA loads of X, Y, Z into rings; one the products: X Y^T, X S
//              and P Z (M = tokens, two accumulators: the row factor f meets X S only) and
//              dS = Y^T Zw (M = channels); two help with the scores' far blocks
//   warps 4-7  scores from TMEM, times D, to bf16 in TMEM (over the scores, as the A operand
//              of P Z); later O from TMEM to global memory, a 128-byte row per thread
//   warps 8-.. one thread per state row (channel): S in fp32 registers, dS from TMEM added,
//              a bf16 copy to shared memory as the B operand of the next chunk's X S
//   warps 12-  w (.) Z as a sum of three bf16 tiles (see below); with 256 channels, where
//              these warps hold the state's second half, the helpers form it
// The products are issued by one thread of a converged warp from descriptors that differ by
// constants: formed anew in a loop they took 180 cycles each, longer than the products.
// The chain from chunk to chunk is dS -> state -> X S, beside it scores -> P -> P Z; the
// loads run ahead by the rings' depth (two tiles of 128 channels of X and of Y).
//
// Precision: P and the copy of S that X S reads are rounded to bf16 (2^-8 of each term, the
// output's own rounding is as large: outputs are 2.3e-3 off where their rounding alone leaves
// 1.7e-3).  P as two bf16 parts, the second over the other half of its scores, gives 1.7e-3 to
// 2.1e-3 and takes 106 us instead of 90 (4 x 37 heads of 2048 tokens of 128 x 128, states read
// and written; 161 instead of 141 for the gradients of 8 x 16 heads of 1024): the split stands
// between the scores and P Z, on every chunk's chain.  For a second part of S there is no shared
// memory with 128 channels.  One part it is.  The carried state is returned in fp32 and lives on
// through every later chunk, so its update must not lose that: Y is exact, and w (.) Z is
// cut into three bf16 values of eight bits each, which is exact.  The three tiles stand side
// by side, so that one product of N = 192 columns reads Y once for all (two with 256
// channels, where TMEM is full: 128 and 64).  lambda^m
// multiplies the state once a chunk, hundreds of times in a long sequence: it is applied as
// a sum of two fp32 numbers.
//
// 64 columns per CTA and not 128: the state and X S shrink, which leaves shared memory for
// two chunks in flight (one at 256 channels), and a batch of few heads fills twice the SMs.
// X Y^T is computed again by every 64 columns; X and Y come from L2.
//
// Measured: 4 x 37 heads x 2048 tokens of 128 x 128 (two CTAs an SM in turn, no states) 86 us; DRAM
// at 37% of its peak, the tensor pipe at 38%, the warps issue in 31% of the cycles.  What bounds a
// chunk is shared memory: the operands of the products (M = 128 by N = 64 reads more bytes a
// product than any other tile here), TMA's writes and the scaled tiles share 128 bytes a
// cycle, and a chunk takes 1.4 times as long as that traffic alone.  Unrolled loops of the
// scaling and of the scores cost more in instruction misses than they save (132 us against
// 94 at one size); two and three issuing warps were slower than one.
#include "decay.h"
#include "decay_plan.h"
#include "tc_common.cuh"
#include "tc_path.h"

namespace gla {
namespace {

constexpr int kC = decay_chunk_tc();  // tokens of a chunk
constexpr int kBV = kDecayTileV;      // columns of V per CTA
constexpr int kThreads = 512;
constexpr int kTmemCols = 512;
// TMEM columns: scores fp32 (then P in bf16), the output accumulators, dS (64 columns for
// each part of Zw; with 256 channels 128 per 128, where the two small parts share theirs)
constexpr uint32_t kColSc = 0, kColOa = 128, kColOb = 192, kColDs = 256;

// Registers a thread, per warpgroup.  Launched with 128; the groups that wait and issue give
// some to those that hold rows of scores and of the state.
template <int KB>
struct Regs {
  static constexpr int roles = 104, rows = 152, state = KB == 1 ? 152 : 128, scale = 104;
  static_assert(roles + rows + (KB == 1 ? state + scale : 2 * state) <= 4 * 128, "more than the launch allocates");
};

// Sets a warpgroup's budget: the instruction that lowers a budget faults on a higher one.
constexpr int kRegsLaunch = 65536 / kThreads;
template <int N>
__device__ __forceinline__ void set_regs() {
  if constexpr (N > kRegsLaunch) dev::regs_inc<N>();
  if constexpr (N < kRegsLaunch) dev::regs_dec<N>();
}

// KB: 128-channel blocks of the contraction
template <int KB>
struct Smem {
  static constexpr int kZStages = KB == 1 ? 2 : 1;
  static constexpr int kTile = kC * 128 * 2;  // 128 channels of X or Y: two SW128 blocks of 64
  static constexpr int kZTile = kC * kBV * 2;
  static constexpr int x = 0, y = x + 2 * kTile, z = y + 2 * kTile, zw = z + kZStages * kZTile, s = zw + 3 * kZTile,
                       t = s + 128 * KB * kBV * 2, bar = t + 528, bytes = bar + 256;
  static_assert(bytes + 1024 <= kMaxDynSmem, "");
};

__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7632); }

// eight bf16 values times f as three bf16 values each, cut (not rounded) so that their sum is the fp32 product
__device__ __forceinline__ void split3(uint4 u, float f, uint4 &zh, uint4 &zm, uint4 &zl) {
  const uint32_t a[4] = {u.x, u.y, u.z, u.w};
  uint32_t h[4], m[4], l[4];
  const dev::f2 f2v = dev::pk(f, f), neg = dev::pk(-1.f, -1.f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const dev::f2 p = dev::mul2(dev::bf16pair(a[j]), f2v);
    float p0, p1;
    dev::upk(p, p0, p1);
    h[j] = high_halves(__float_as_uint(p0), __float_as_uint(p1));
    const dev::f2 q = dev::fma2(dev::bf16pair(h[j]), neg, p);
    dev::upk(q, p0, p1);
    m[j] = high_halves(__float_as_uint(p0), __float_as_uint(p1));
    const dev::f2 r = dev::fma2(dev::bf16pair(m[j]), neg, q);
    dev::upk(r, p0, p1);
    l[j] = high_halves(__float_as_uint(p0), __float_as_uint(p1));
  }
  zh = make_uint4(h[0], h[1], h[2], h[3]);
  zm = make_uint4(m[0], m[1], m[2], m[3]);
  zl = make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ void st_global_32(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ void ld_global_32(const float *p, float *x) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(p)
               : "memory");
}

// ACC: a contraction taken in pieces, with partial outputs read or written
template <int KB, bool OUT, bool REV, bool ACC>
__global__ void __launch_bounds__(kThreads, 1)
    k_decay_tc(const __grid_constant__ DecayWalk w, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ) {
  using L = Smem<KB>;
  constexpr int NZ = L::kZStages;
  constexpr int kStateWarps = 4 * KB;
  // warps of the first warpgroup: a helper reads the rows (TMEM lanes) of its number mod 4,
  // and the rows that need one are the last 64, in a reverse walk the first
  constexpr int kLoadWarp = REV ? 2 : 0, kIssueWarp = kLoadWarp + 1, kHelp0 = REV ? 0 : 2;
  constexpr int kScale0 = KB == 1 ? 12 : kHelp0, kScaleWarps = KB == 1 ? 4 : 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float *W = (float *)(smem + L::t);  // W[n] = lambda^n, n = 0 .. 128
  uint64_t *bars = (uint64_t *)(smem + L::bar);
  // slot (i KB + kb) mod 2 of X and Y holds channel block kb of chunk i
  uint64_t *xfull = bars, *xempty = xfull + 2, *yfull = xempty + 2, *yempty = yfull + 2, *zfull = yempty + 2,
           *zempty = zfull + 2, *scfull = zempty + 2, *pfull = scfull + 1, *ofull = pfull + 1, *oempty = ofull + 1,
           *dsfull = oempty + 1, *dsempty = dsfull + 1, *sfull = dsempty + 1, *qsdone = sfull + 1, *zready = qsdone + 1,
           *done = zready + 1;
  uint32_t *tslot = (uint32_t *)(done + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (w.V + kBV - 1) / kBV;
  const uint32_t line = blockIdx.x / (uint32_t)tiles;
  const int vt = (int)(blockIdx.x - line * (uint32_t)tiles), seg = blockIdx.y;
  const long bh = line;
  const int b = (int)(line / (uint32_t)w.H), h = (int)(line - (uint32_t)b * (uint32_t)w.H), v0 = vt * kBV;
  const int kz = OUT ? 0 : blockIdx.z;  // without outputs, 128 channels a CTA: the first block of these
  if (tid == 32 * kLoadWarp) {
    dev::prefetch_tmap(&tmY);
    dev::prefetch_tmap(&tmZ);
    if (OUT) dev::prefetch_tmap(&tmX);
    for (int i = 0; i < 12; ++i) dev::mbar_init(&xfull[i], 1);
    dev::mbar_init(scfull, 1);
    dev::mbar_init(pfull, 6);
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
  // what the set-up reads from memory is asked for at once
  const float ld = __ldg(w.ld + h);
  const dev::DSeq sq = dev::decay_seq(w, b);
  const int n = (sq.len + kC - 1) / kC, nseg = max(1, (n + w.L - 1) / w.L);
  if (seg >= nseg || (!OUT && seg == nseg - 1)) {  // the whole CTA
    if (!OUT && w.pre_join && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) dev::pdl_wait();
    return;
  }
  if (OUT && w.wait_first) dev::pdl_wait();
  if (!OUT || w.lead) dev::pdl_launch_dependents();
  const int c_begin = seg * w.L, nloc = max(0, min(n, c_begin + w.L) - c_begin);
  auto chunk_of = [&](int i) { return REV ? n - 1 - (c_begin + i) : c_begin + i; };
  auto live_of = [&](int i) { return min(kC, sq.len - chunk_of(i) * kC); };
  const int ksteps = (w.K + 15) / 16, kblocks = (w.K + 63) / 64;
  // of channel block kb: 16-channel steps, 64-column blocks
  auto ksteps_of = [&](int kb) { return min(8, ksteps - 8 * kb); };
  auto kblocks_of = [&](int kb) { return max(0, min(2, kblocks - 2 * (kz + kb))); };
  auto slot = [&](int i, int kb) { return (i * KB + kb) & 1; };
  auto phase = [&](int i, int kb) { return (uint32_t)(((i * KB + kb) >> 1) & 1); };
  // the coordinate along an axis: a tensor shared along it (distance 0) has one entry there
  auto axis = [](long distance, int c) { return distance ? c : 0; };
  auto load_y = [&](int i, int kb) {
    const int s = slot(i, kb), row = (int)(sq.row0 + (long)chunk_of(i) * kC);
    dev::mbar_arrive_expect_tx(&yfull[s], (uint32_t)(kblocks_of(kb) * kC * 128));
    for (int cb = 0; cb < kblocks_of(kb); ++cb)
      dev::tma_load_4d(smem + L::y + s * L::kTile + cb * kC * 128, &tmY, 128 * (kz + kb) + cb * 64, row, axis(w.y.sh, h), axis(w.y.sb, sq.b),
                       &yfull[s]);
  };
  auto load_x = [&](int i, int kb) {
    const int s = slot(i, kb), row = (int)(sq.row0 + (long)chunk_of(i) * kC);
    dev::mbar_arrive_expect_tx(&xfull[s], (uint32_t)(kblocks_of(kb) * kC * 128));
    for (int cb = 0; cb < kblocks_of(kb); ++cb)
      dev::tma_load_4d(smem + L::x + s * L::kTile + cb * kC * 128, &tmX, 128 * kb + cb * 64, row, axis(w.x.sh, h), axis(w.x.sb, sq.b),
                       &xfull[s]);
  };
  auto load_z = [&](int i) {
    const int s = i % NZ, row = (int)(sq.row0 + (long)chunk_of(i) * kC);
    dev::mbar_arrive_expect_tx(&zfull[s], (uint32_t)L::kZTile);
    dev::tma_load_4d(smem + L::z + s * L::kZTile, &tmZ, v0, row, axis(w.z.sh, h), axis(w.z.sb, sq.b), &zfull[s]);
  };
  if (tid == 32 * kLoadWarp && nloc > 0) {  // the first chunk's loads run beside the set-up
    for (int kb = 0; kb < KB; ++kb) {
      if (OUT) load_x(0, kb);
      load_y(0, kb);
    }
    load_z(0);
  }
  if (warp == kIssueWarp) dev::tmem_alloc(tslot, kTmemCols);
  const double rate = dev::decay_rate(ld, w.status);
  if (tid >= 128 && tid <= 128 + kC) W[tid - 128] = (float)dev::decay_pow(rate, tid - 128);
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tmem = *tslot;
  using R = Regs<KB>;

  // ============================ w (.) Z ============================
  // w (.) Z of chunk i
  const int t0 = tid - 32 * kScale0;
  constexpr int kStep = 32 * kScaleWarps, kIter = kC * 8 / kStep;  // 16-byte units per pass, passes
  auto scale_z = [&](int i, bool &ok) {
    const int s = i % NZ;
    const int m = live_of(i);
    if (ok) ok = dev::mbar_wait(&zfull[s], (uint32_t)((i / NZ) & 1), w.status);
    uint8_t *zt = smem + L::z + s * L::kZTile, *zw = smem + L::zw;
    // a row is eight 16-byte units; their place in the swizzled row does not matter here
    if (ok && m == kC) {
      if (i > 0) ok = dev::mbar_wait(dsfull, (uint32_t)((i - 1) & 1), w.status);
#pragma unroll 1
      for (int j = 0; j < kIter; j += 2) {
        const int e = 16 * (t0 + j * kStep), r = (t0 + j * kStep) >> 3;
        const uint4 u0 = *reinterpret_cast<const uint4 *>(zt + e), u1 = *reinterpret_cast<const uint4 *>(zt + e + 16 * kStep);
        const float f0 = W[REV ? r + 1 : kC - 1 - r], f1 = W[REV ? r + kStep / 8 + 1 : kC - 1 - kStep / 8 - r];
        uint4 zh, zm, zl;
        split3(u0, f0, zh, zm, zl);
        *reinterpret_cast<uint4 *>(zw + e) = zh;
        *reinterpret_cast<uint4 *>(zw + L::kZTile + e) = zm;
        *reinterpret_cast<uint4 *>(zw + 2 * L::kZTile + e) = zl;
        split3(u1, f1, zh, zm, zl);
        *reinterpret_cast<uint4 *>(zw + e + 16 * kStep) = zh;
        *reinterpret_cast<uint4 *>(zw + L::kZTile + e + 16 * kStep) = zm;
        *reinterpret_cast<uint4 *>(zw + 2 * L::kZTile + e + 16 * kStep) = zl;
      }
    } else if (ok) {
      // Rows behind the sequence hold anything, and zero times it must not be NaN: Y's are
      // cleared (X Y^T of this chunk waits for it), and so are those of Z that the products read.
      const int m16 = (m + 15) & ~15;
      if (i > 0) ok = dev::mbar_wait(dsfull, (uint32_t)((i - 1) & 1), w.status);
#pragma unroll 1
      for (int u = t0; u < m16 * 8; u += kStep) {
        const int r = u >> 3, e = 16 * u;
        uint4 zh, zm, zl, a = *reinterpret_cast<const uint4 *>(zt + e);
        if (r >= m) {
          a = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(zt + e) = a;
        }
        split3(a, W[r < m ? (REV ? r + 1 : m - 1 - r) : 0], zh, zm, zl);
        *reinterpret_cast<uint4 *>(zw + e) = zh;
        *reinterpret_cast<uint4 *>(zw + L::kZTile + e) = zm;
        *reinterpret_cast<uint4 *>(zw + 2 * L::kZTile + e) = zl;
      }
      const int dead = (kC - m) * 8;
      for (int kb = 0; kb < KB; ++kb) {
        const int sy = slot(i, kb);
        if (ok) ok = dev::mbar_wait(&yfull[sy], phase(i, kb), w.status);
        if (!ok) break;
#pragma unroll 1
        for (int u = t0; u < dead * kblocks_of(kb); u += kStep)
          *reinterpret_cast<uint4 *>(smem + L::y + sy * L::kTile + (u / dead) * kC * 128 + m * 128 + (u % dead) * 16) =
              make_uint4(0, 0, 0, 0);
      }
    }
    dev::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(zready);
  };

  // ============================ P ============================
  // Row t of P = (X Y^T) (.) D, 32 columns (tokens j = 32 jb + e) a block; a block of P lies
  // over the first half of its own scores.  On the diagonal the weights are kept in
  // registers; beside it they are multiplied on from the block's near end, lambda a column,
  // where `near` is this row's weight: a table in shared memory would wait for the
  // products, whose operands take all its bandwidth.
  const float lam1 = W[1];
  const dev::f2 lam2 = dev::pk(W[2], W[2]), lam8 = dev::pk(W[8], W[8]);
  auto store_p = [&](uint32_t base, const float *sc, int jb) {
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) p[e] = dev::pack_bf16(sc[2 * e], sc[2 * e + 1]);
    dev::tmem_st16u(base + kColSc + 32 * jb, p);
  };
  auto weigh = [&](float *sc, float near) {
    dev::f2 f[4];  // four pairs of columns in turn
    f[0] = REV ? dev::pk(near, near * lam1) : dev::pk(near * lam1, near);
#pragma unroll
    for (int k = 1; k < 4; ++k) f[k] = dev::mul2(f[k - 1], lam2);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float *x = sc + (REV ? 2 * k : 30 - 2 * k);
      dev::upk(dev::mul2(dev::pk(x[0], x[1]), f[k & 3]), x[0], x[1]);
      if (k < 12) f[k & 3] = dev::mul2(f[k & 3], lam8);
    }
  };
  // the helpers' share: two blocks away from the diagonal
  auto help_p = [&](int i, bool &ok) {
    const int q4 = warp & 3, t = 32 * q4 + lane, jb0 = REV ? 2 : 0;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q4) << 16);
    if (ok) ok = dev::mbar_wait(scfull, (uint32_t)(i & 1), w.status);
    dev::tc_fence_after();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float sc[32];
      dev::tmem_ld32(lane_base + kColSc + 32 * (jb0 + u), sc);
      const float near = W[REV ? 32 * (jb0 + u) - t : t - 32 * (jb0 + u) - 31];
      dev::tmem_wait_ld();
      weigh(sc, near);
      store_p(lane_base, sc, jb0 + u);
    }
    dev::tmem_wait_st();
    dev::tc_fence_before();
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(pfull);
  };

  if (warp < 4) {
    set_regs<R::roles>();
    if (warp == kLoadWarp) {
      // ============================ loads ============================
      if (lane == 0 && nloc > 0) {
        bool ok = true;
        // the next tile of each kind that has not been issued: (chunk, block)
        int ni = 1;  // chunks 0 .. ni - 1 are issued
        int xl = KB, yl = KB, zl = 1;
        for (; ni < nloc && ok; ++ni) {
          for (int kb = 0; kb < KB && ok; ++kb) {
            const int s = slot(ni, kb);
            if (OUT) {
              if (ni * KB + kb >= 2) ok = dev::mbar_wait(&xempty[s], phase(ni, kb) ^ 1u, w.status);
              if (!ok) break;
              load_x(ni, kb);
              ++xl;
            }
          }
          for (int kb = 0; kb < KB && ok; ++kb) {
            const int s = slot(ni, kb);
            if (ni * KB + kb >= 2) ok = dev::mbar_wait(&yempty[s], phase(ni, kb) ^ 1u, w.status);
            if (!ok) break;
            load_y(ni, kb);
            ++yl;
          }
          if (ok && ni >= NZ) ok = dev::mbar_wait(&zempty[ni % NZ], (uint32_t)((ni / NZ - 1) & 1), w.status);
          if (!ok) break;
          load_z(ni);
          ++zl;
        }
        // every load issued lands before the CTA ends, also where a wait ran out
        for (int j = max(0, yl - 2); j < yl; ++j) (void)dev::mbar_wait(&yfull[j & 1], (uint32_t)((j >> 1) & 1), w.status);
        if (OUT)
          for (int j = max(0, xl - 2); j < xl; ++j) (void)dev::mbar_wait(&xfull[j & 1], (uint32_t)((j >> 1) & 1), w.status);
        for (int j = max(0, zl - NZ); j < zl; ++j) (void)dev::mbar_wait(&zfull[j % NZ], (uint32_t)((j / NZ) & 1), w.status);
      }
    } else if (warp == kIssueWarp) {
      // ============================ products ============================
      // the whole warp runs the loop (all of it is warp-uniform), one thread issues
      constexpr uint32_t id_sc = dev::idesc_bf16(kC, kC, false, false);   // X, Y: K-major
      constexpr uint32_t id_o = dev::idesc_bf16(kC, kBV, false, true);    // X or P (TMEM); S or Z: MN-major
      constexpr uint32_t id_dh = dev::idesc_bf16(128, (KB == 1 ? 3 : 2) * kBV, true, true);  // Y, parts of Zw: MN-major
      constexpr uint32_t id_dl = dev::idesc_bf16(128, kBV, true, true);
      // descriptors of a tile's first step; step kk lies koff(kk) (K-major) or mnoff(kk) further
      const uint64_t dX = dev::desc_kmajor(dev::smem_u32(smem + L::x), kC, 0, 0),
                     dYk = dev::desc_kmajor(dev::smem_u32(smem + L::y), kC, 0, 0),
                     dYm = dev::desc_mnmajor(dev::smem_u32(smem + L::y), kC, 0, 0),
                     dZ = dev::desc_mnmajor(dev::smem_u32(smem + L::z), kC, 0, 0),
                     dS = dev::desc_mnmajor(dev::smem_u32(smem + L::s), 128 * KB, 0, 0),
                     dZw = dev::desc_mnmajor(dev::smem_u32(smem + L::zw), kC, 0, 0);
      constexpr auto koff = [](int kk) { return (uint64_t)(((kk >> 2) * kC * 128 + (kk & 3) * 32) >> 4); };
      constexpr auto mnoff = [](int kk) { return (uint64_t)((kk * 16 * 128) >> 4); };
      constexpr uint64_t kTileD = L::kTile >> 4, kZTileD = L::kZTile >> 4;
      const bool leader = dev::elect_one();
      auto wait = [&](uint64_t *bar, uint32_t par) { return __all_sync(0xffffffffu, dev::mbar_wait(bar, par, w.status)) != 0; };
      bool ok = true;
      // The first tiles of chunk i are looked at before the wait for P of the chunk before, so
      // that X Y^T follows P Z without a pause.
      auto tiles_of = [&](int i) {
        ok = ok && wait(&xfull[slot(i, 0)], phase(i, 0)) && wait(&yfull[slot(i, 0)], phase(i, 0));
      };
      // X Y^T of chunk i
      auto scores = [&](int i) {
        if (live_of(i) < kC) ok = ok && wait(zready, (uint32_t)(i & 1));  // Y's rows behind the sequence are cleared
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const int s = slot(i, kb);
          if (KB == 2) ok = ok && wait(&xfull[s], phase(i, kb)) && wait(&yfull[s], phase(i, kb));
          if (!ok) return;
          dev::tc_fence_after();
          const int ks = ksteps_of(kb);
          const uint64_t x = dX + s * kTileD, y = dYk + s * kTileD;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              if (kk < ks) dev::umma_bf16(tmem + kColSc, x + koff(kk), y + koff(kk), id_sc, kb + kk > 0 ? 1u : 0u);
            if (kb == KB - 1) dev::umma_commit(scfull);
          }
          __syncwarp();
        }
      };
      // X S of chunk i
      auto inter = [&](int i) {
        ok = ok && wait(sfull, (uint32_t)(i & 1));
        if (ok && i > 0) ok = wait(oempty, (uint32_t)((i & 1) ^ 1));
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const int s = slot(i, kb);
          if (!ok) return;
          dev::tc_fence_after();
          const int ks = ksteps_of(kb);
          const uint64_t x = dX + s * kTileD;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              if (kk < ks) dev::umma_bf16(tmem + kColOb, x + koff(kk), dS + mnoff(8 * kb + kk), id_o, kb + kk > 0 ? 1u : 0u);
            dev::umma_commit(&xempty[s]);  // X Y^T came first
            if (kb == KB - 1) dev::umma_commit(qsdone);
          }
          __syncwarp();
        }
      };
      if (OUT && KB == 1 && nloc > 0) tiles_of(0);
      for (int i = 0; i < nloc && ok; ++i) {
        const uint32_t par = (uint32_t)(i & 1);
        const int ts = (live_of(i) + 15) / 16;  // 16-token steps that hold a live token
        // X S goes behind dS with 128 channels: the state that it reads is made from dS of the
        // chunk before, and P is ready by then.  With 256 it goes before dS, so that the next
        // X, which has no second buffer, arrives while dS is formed.
        if (OUT) scores(i);
        if (OUT && KB == 2) inter(i);
        ok = ok && wait(zready, par);  // (the warps that arrive there have waited for Z)
        if (ok && i > 0) ok = wait(dsempty, par ^ 1u);
        if (!ok) break;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const int s = slot(i, kb);
          if (!OUT) ok = ok && wait(&yfull[s], phase(i, kb));
          if (!ok) break;
          dev::tc_fence_after();
          const uint64_t y = dYm + s * kTileD;
          const uint32_t d = tmem + kColDs + kb * 128;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              if (kk < ts) {
                dev::umma_bf16(d, y + mnoff(kk), dZw + mnoff(kk), id_dh, kk > 0 ? 1u : 0u);
                if (KB == 2) dev::umma_bf16(d + kBV, y + mnoff(kk), dZw + 2 * kZTileD + mnoff(kk), id_dl, 1u);
              }
            dev::umma_commit(&yempty[s]);
            if (kb == KB - 1) dev::umma_commit(dsfull);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (OUT && KB == 1) inter(i);
        if (!ok) break;
        if (OUT) {
          if (KB == 1 && i + 1 < nloc) tiles_of(i + 1);
          ok = ok && wait(pfull, par);
          if (!ok) break;
          dev::tc_fence_after();
        }
        if (leader) {
          const uint64_t z = dZ + (i % NZ) * kZTileD;
          if (OUT) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              if (kk < ts) dev::umma_bf16_ts(tmem + kColOa, tmem + kColSc + 32 * (kk >> 1) + 8 * (kk & 1), z + mnoff(kk), id_o, kk > 0 ? 1u : 0u);
            dev::umma_commit(ofull);
          }
          dev::umma_commit(&zempty[i % NZ]);
        }
        __syncwarp();
      }
      if (leader) {
        dev::umma_commit(done);  // all products have completed before TMEM is released
        (void)dev::mbar_wait(done, 0, w.status);
      }
      __syncwarp();
    } else {
      bool ok = true;
      for (int i = 0; i < nloc; ++i) {
        if (KB == 2) scale_z(i, ok);
        if (OUT) help_p(i, ok);
      }
    }
  } else if (warp < 8) {
    // ============================ P and O ============================
    set_regs<R::rows>();
    if (OUT) {
      const int q4 = warp & 3, t = 32 * q4 + lane;
      const uint32_t lane_base = tmem + ((uint32_t)(32 * q4) << 16);
      const long rows = w.packed ? w.T : (long)w.nseq * w.T;
      const bool wide = (((uintptr_t)w.o.p | (uintptr_t)(2 * w.o.st) | (uintptr_t)(2 * w.o.sh) | (uintptr_t)(2 * w.o.sb)) & 31u) == 0;
      const int nv = min(kBV, w.V - v0);  // a multiple of 8
      const int jo = q4 ^ 1;  // the block beside the diagonal's: on the near or the far side
      const bool beside = REV ? (q4 & 1) == 0 : (q4 & 1) == 1;
      const bool clear = REV ? q4 >= 2 : q4 < 2;  // the other two blocks: zero, or a helper's
      const float near = W[REV ? 32 - lane : lane + 1];
      float fd[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int g = REV ? e - lane : lane - e;
        fd[e] = g >= 0 ? W[g] : 0.f;
      }
      bool ok = true;
      for (int i = 0; i < nloc; ++i) {
        const uint32_t par = (uint32_t)(i & 1);
        const int m = live_of(i);
        const long row0 = sq.row0 + (long)chunk_of(i) * kC;
        if (ok) ok = dev::mbar_wait(scfull, par, w.status);
        dev::tc_fence_after();
        float sc[32];
        dev::tmem_ld32(lane_base + kColSc + 32 * q4, sc);
        dev::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          dev::upk(dev::mul2(dev::pk(sc[e], sc[e + 1]), dev::pk(fd[e], fd[e + 1])), sc[e], sc[e + 1]);
        store_p(lane_base, sc, q4);
        if (beside) {
          dev::tmem_ld32(lane_base + kColSc + 32 * jo, sc);
          dev::tmem_wait_ld();
          weigh(sc, near);
          store_p(lane_base, sc, jo);
        } else {
          const uint32_t zero[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
          dev::tmem_st16u(lane_base + kColSc + 32 * jo, zero);
        }
        if (clear) {
          const uint32_t zero[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
          dev::tmem_st16u(lane_base + kColSc + 32 * (REV ? 0 : 2), zero);
          dev::tmem_st16u(lane_base + kColSc + 32 * (REV ? 1 : 3), zero);
        }
        dev::tmem_wait_st();
        dev::tc_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(pfull);

        if (ok) ok = dev::mbar_wait(ofull, par, w.status);
        dev::tc_fence_after();
        const float f = W[t < m ? (REV ? m - 1 - t : t + 1) : 0];
        __nv_bfloat16 *o = (__nv_bfloat16 *)w.o.p + sq.b * w.o.sb + h * w.o.sh + (row0 + t) * w.o.st + v0;
        const bool live = t < m && ok;
#pragma unroll 1
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
          const dev::f2 f2v = dev::pk(f, f);
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            dev::upk(dev::fma2(f2v, dev::pk(c[e], c[e + 1]), dev::pk(a[e], a[e + 1])), a[e], a[e + 1]);
          if (ACC && live) {
            const long row = w.packed ? row0 + t : (long)b * w.T + row0 + t;
            float *part = w.acc + ((long)h * rows + row) * w.V + v0 + 32 * hf;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if (32 * hf + e < nv) {
                float4 x = make_float4(a[e], a[e + 1], a[e + 2], a[e + 3]);
                if (w.acc_in) {
                  const float4 y = *reinterpret_cast<const float4 *>(part + e);
                  x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                  a[e] = x.x, a[e + 1] = x.y, a[e + 2] = x.z, a[e + 3] = x.w;
                }
                if (w.acc_out) *reinterpret_cast<float4 *>(part + e) = x;
              }
          }
          uint32_t r[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) r[e] = dev::pack_bf16(a[2 * e], a[2 * e + 1]);
          if (!live || (ACC && w.acc_out)) continue;
          if (wide && nv == kBV) {
            st_global_32(o + 32 * hf, r);
            st_global_32(o + 32 * hf + 16, r + 8);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (32 * hf + 8 * j < nv)
                *reinterpret_cast<uint4 *>(o + 32 * hf + 8 * j) =
                    make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
          }
        }
      }
    }
  } else if (warp < 8 + kStateWarps) {
    // ============================ state ============================
    set_regs<R::state>();
    const int q4 = warp & 3, kb = (warp - 8) >> 2, kc = 128 * kb + 32 * q4 + lane, kr = 128 * kz + kc;  // this thread's channel (of the CTA's, of all)
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q4) << 16);
    const long KV = (long)w.K * w.V;
    float *wsb = w.ws + bh * w.P * KV + (long)kr * w.V + v0;
    const bool kok = kr < w.K;
    const int nv = min(kBV, w.V - v0);  // a multiple of 8
    const bool pass = w.P > 1 && nseg > 1;
    int i0, i1;
    dev::decay_slots<true>(w.s0, w.s1, w.alias, w.nseq, b, OUT ? w.status : nullptr, i0, i1);
    float S[kBV];
#pragma unroll
    for (int e = 0; e < kBV; ++e) S[e] = 0.f;
    if (kok) {
      if (OUT && pass) {
        if (!w.settled) dev::pdl_wait();
        // entry 0: the start state (segment 0); entries 1 .. seg: states of the segments before
        // lambda^(tokens of a segment) as a sum, like lambda^m below
        const double across = dev::decay_pow(rate, (long)w.L * kC);
        const float far = (float)across, rest = (float)(across - (double)far);
        for (int j = seg == 0 ? 0 : 1; j <= seg; ++j) {
          const float *u = wsb + j * KV;
#pragma unroll
          for (int e = 0; e < kBV; e += 4)
            if (e < nv) {
              const float4 x = *reinterpret_cast<const float4 *>(u + e);
              S[e] = fmaf(S[e], far, fmaf(S[e], rest, x.x));
              S[e + 1] = fmaf(S[e + 1], far, fmaf(S[e + 1], rest, x.y));
              S[e + 2] = fmaf(S[e + 2], far, fmaf(S[e + 2], rest, x.z));
              S[e + 3] = fmaf(S[e + 3], far, fmaf(S[e + 3], rest, x.w));
            }
        }
      } else if (seg == 0) {
        if (i0 >= 0) {
          const float *u = w.s0.p + i0 * w.s0.slot + h * w.s0.head + kr * w.s0.row + v0 * w.s0.col;
          if (w.s0.col == 1 && ((uintptr_t)u & 31u) == 0) {
#pragma unroll
            for (int e = 0; e < kBV; e += 8)
              if (e < nv) ld_global_32(u + e, S + e);
          } else if (w.s0.col == 1) {
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
    const uint32_t srow = dev::smem_u32(smem + L::s) + (uint32_t)kc * 128u;
    auto publish = [&]() {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dev::st_shared_v4(srow + (uint32_t)((j ^ (kc & 7)) << 4), dev::pack_bf16(S[8 * j], S[8 * j + 1]),
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
      // 16 columns at a time, all of their parts in one trip; the small ones are added first
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float d0[16], d1[16], d2[16];
        const uint32_t c = lane_base + kColDs + kb * 128 + 16 * g;
        dev::tmem_ld16(c, d0);
        dev::tmem_ld16(c + kBV, d1);
        if (KB == 1) dev::tmem_ld16(c + 2 * kBV, d2);
        dev::tmem_wait_ld();
        if (g == 3) {
          dev::tc_fence_before();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(dsempty);
        }
        const dev::f2 dh2 = dev::pk(dh, dh), dl2 = dev::pk(dl, dl);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          float *x = S + 16 * g + e;
          const dev::f2 old = dev::pk(x[0], x[1]);
          dev::f2 lo = dev::pk(d1[e], d1[e + 1]);
          if (KB == 1) lo = dev::add2(lo, dev::pk(d2[e], d2[e + 1]));
          lo = dev::add2(dev::fma2(old, dl2, lo), dev::pk(d0[e], d0[e + 1]));
          dev::upk(dev::fma2(old, dh2, lo), x[0], x[1]);
        }
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
        if (w.s1.col == 1 && ((uintptr_t)u & 31u) == 0) {
#pragma unroll
          for (int e = 0; e < kBV; e += 8)
            if (e < nv) st_global_32(u + e, reinterpret_cast<const uint32_t *>(S + e));
        } else if (w.s1.col == 1) {
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
  } else {
    set_regs<R::scale>();
    bool ok = true;
    for (int i = 0; i < nloc; ++i) scale_z(i, ok);
  }
  dev::tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) dev::tmem_dealloc(tmem, kTmemCols);
  if ((OUT ? w.follows() : w.pre_join) && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) dev::pdl_wait();
}

// ---------------------------------------------------------------- host

bool ok_view(const DView &v, const DecayWalk &w) {
  // TMA: 16-byte base and distances below 2^40 bytes, that of tokens not zero; heads or
  // sequences that share a tensor (distance 0) are an axis of one entry
  const bool dense = !w.packed && w.nseq > 1;
  auto fits = [](long s, bool used) { return !used || (s % 8 == 0 && s < (1L << 38)); };
  return ((uintptr_t)v.p & 15u) == 0 && fits(v.st, w.T > 1) && (v.st > 0 || w.T == 1) && fits(v.sh, w.H > 1) &&
         fits(v.sb, dense);
}

bool make_map(CUtensorMap *m, const DView &v, const DecayWalk &w, int channels) {
  const bool heads = w.H > 1 && v.sh, batch = !w.packed && w.nseq > 1 && v.sb;
  auto step = [](long s, bool used) { return (uint64_t)(used ? 2 * s : 16); };
  const uint64_t dims[4] = {(uint64_t)channels, (uint64_t)w.T, (uint64_t)(heads ? w.H : 1), (uint64_t)(batch ? w.nseq : 1)};
  const uint64_t strides[3] = {step(v.st, w.T > 1), step(v.sh, heads), step(v.sb, batch)};
  return tc::map4_bf16(m, v.p, dims, strides, 64, kC);
}

// A kernel's shared memory, set once per device.
template <auto kernel>
int prepare(int smem) {
  static DeviceSlots slots;
  const int e = per_device(slots, [smem] {
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r != cudaSuccess) note_cuda_error(r);
    return r == cudaSuccess ? 1 : -1;
  });
  return e == 1 ? GLA_OK : GLA_ERR_CUDA;
}

template <int KB, bool REV, bool ACC>
int launch(const DecayWalk &w, cudaStream_t st) {
  CUtensorMap mx, my, mz;
  if (!make_map(&mx, w.x, w, w.K) || !make_map(&my, w.y, w, w.K) || !make_map(&mz, w.z, w, w.V)) return GLA_ERR_CUDA;
  const unsigned gx = (unsigned)((long)w.nseq * w.H * ((w.V + kBV - 1) / kBV));
  if (w.P > 1 && (w.stage & 1)) {
    // the states of 128 channels do not meet those of the others before the outputs
    constexpr int smem = Smem<1>::bytes + 1024;
    if (const int e = prepare<k_decay_tc<1, false, REV, false>>(smem)) return e;
    const dim3 grid(gx, w.P - 1, w.K > 128 ? 2 : 1);
    if (w.pre_join)
      GLA_LAUNCH(K_DECAY_STATES, st,
                 (void)launch_pdl(k_decay_tc<1, false, REV, false>, grid, dim3(kThreads), smem, st, w, mx, my, mz));
    else
      GLA_LAUNCH(K_DECAY_STATES, st, (k_decay_tc<1, false, REV, false><<<grid, kThreads, smem, st>>>(w, mx, my, mz)));
  }
  if (!(w.stage & 2)) return GLA_OK;
  constexpr int smem = Smem<KB>::bytes + 1024;
  if (const int e = prepare<k_decay_tc<KB, true, REV, ACC>>(smem)) return e;
  if (w.follows())
    GLA_LAUNCH(K_DECAY_WALK, st,
               (void)launch_pdl(k_decay_tc<KB, true, REV, ACC>, dim3(gx, w.P), dim3(kThreads), smem, st, w, mx, my, mz));
  else
    GLA_LAUNCH(K_DECAY_WALK, st, (k_decay_tc<KB, true, REV, ACC><<<dim3(gx, w.P), kThreads, smem, st>>>(w, mx, my, mz)));
  return GLA_OK;
}

}  // namespace

bool decay_tc_takes(const DecayWalk &w, int dtype) {
  return dtype == GLA_DTYPE_BF16 && w.K % 8 == 0 && w.V % 8 == 0 && ok_view(w.x, w) && ok_view(w.y, w) &&
         ok_view(w.z, w) && ok_view(w.o, w);
}

int decay_walk_tc(const DecayWalk &w, cudaStream_t st) {
  if (w.acc_in || w.acc_out) return w.reverse ? launch<2, true, true>(w, st) : launch<2, false, true>(w, st);
  if (w.reverse) return w.K <= 128 ? launch<1, true, false>(w, st) : launch<2, true, false>(w, st);
  return w.K <= 128 ? launch<1, false, false>(w, st) : launch<2, false, false>(w, st);
}

}  // namespace gla
