// sgr_kv_attn_rows.cuh -- attention over the paged E4M3 cache for many query
// rows a key/value head (chunks of a prompt):
//
//     o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q.k_t)
//
// Per row tile (256 rows, two halves j of 128) and 128-token tile of the cache:
//
//     S_j [128 rows, 128 tokens] = Q_j K^T    FP8: K's codes as they are, Q = hi + lo
//     P_j = 2^(S' - R), FP16                  two threads a row, 64 tokens each
//     O_j [128 rows, D]         += P_j V      FP16: P from tensor memory, V widened
//
// Q's parts hi = e4m3(b), lo = e4m3(b - hi) go into one accumulator; with the
// row's largest |b| in [128, 256) they hold all 8 bits of a BF16 query down to
// 2^-9 of it and an absolute 2^-18 below.  Splitting P the same way costs
// three conversions for two weights, and conversions share the exponential
// unit's 16 lanes a cycle: 2560 cycles a 128 x 128 tile against 1024 for the
// exponentials alone (two chunks of some 600 tokens over 6007: 190 us with the
// weights in two parts, 129 without).  So V is widened to FP16 instead (exact), once for
// both halves, with integer instructions, and P is an FP16 weight: 11 bits
// down to 2^-22 of the largest.
//
// R, a whole number, is a row's first maximum rounded up and moves when a score
// exceeds it by more than FP16 holds (2^7.5 times); then the sum and the row's
// accumulator (in tensor memory) are rescaled by a power of two.  The row's two
// threads agree on it by a vote of their two warps a tile.  The weights
// overwrite the scores' columns.
//
// Bound: the chain of a half: its weights (2000 cycles a tile), then their
// product, its completion and the next scores (2100; the scores' columns are
// the weights', so these products cannot overlap), with the other half half a
// turn behind.  Tensor memory is full (two halves of scores and outputs, 128
// columns each): a third chain would take scores of fewer tokens at a time.  Measured for two chunks of some
// 600 tokens over 6007 (28 heads over 4, 74 GFLOP): 118 us, 625 TFLOP/s,
// tensor pipe 31% and issue slots 58% of active cycles; with one softmax
// thread a row instead of two 129 us.
//
// Roles (704 threads, one CTA an SM): warps 0-7 and 8-15 softmax of the halves
// (and their query operands), 16-19 widen V, warp 20 walks the work and loads
// pages, warp 21 issues the MMAs.
#pragma once

#include "sgr_kv_attn.cuh"

namespace sgr {

constexpr int kRowsNT = 256, kRowsThreads = 704;

template <int D>
struct RowsCtl {
  static constexpr int kStages = 2, kMeta = 4, S = kStages, M = kMeta;
  static constexpr bool kStopStage = true;
  uint64_t kfull[S], vfull[S], empty[S];
  uint64_t sfull[2], pfull[2], pvdone[2], wfull[2], wempty[2], qfull[2], drain;
  uint64_t segfull[kAttnQueue], segempty[kAttnQueue];
  uint32_t tmem;
  int abort;
  int go[2][2];
  AttnSeg seg[kAttnQueue];
  // of a tile (the softmax warps may be two tiles behind the copies)
  float kscale[M][8], vexp[M][8];
  int flags[M], live[M][2];
  float qf[kRowsNT];
  float pair[2][2][128];  // of a row's two threads: maxima, sums of weights
  unsigned nan_tokens[2][4];           // of the widened tile: tokens with a NaN value
  uint32_t nan_mask[2][kAttnTile][4];  // and which of its elements
};

template <int D>
constexpr int rows_ctl_bytes() {
  return (int)((sizeof(RowsCtl<D>) + 1023) / 1024 * 1024);
}

// Ring, query operands (hi and lo of both halves), two widened value tiles.
template <int D>
constexpr int rows_attn_smem_bytes() {
  return 1024 + rows_ctl_bytes<D>() + RowsCtl<D>::kStages * 2 * kAttnTile * D + 2 * kRowsNT * D + 2 * kAttnTile * D * 2;
}

// 32 columns of the warp's lanes; the registers hold them after the wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// D (+)= A[tmem] . B[smem] with FP16 operands: A as in mma_bf16_tmem_a.
constexpr uint32_t idesc_f16_f32(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Two codes (a 16-bit pair in the low half of x) to FP16, on the integer and
// FP16 units; NaN codes read as 480.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t widen2(uint32_t x) {
  uint32_t t, r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(t) : "r"(x), "n"(SEL));  // codes in the low bytes, signs above
  t = (t << 7) & 0xBF80BF80u;                                   // the value times 2^-8
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(0x5C005C00u));  // 0x5C00 = 256
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads, 1)
    kv_attn_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const AttnParams p) {
  constexpr int S = RowsCtl<D>::kStages, M = RowsCtl<D>::kMeta, kTile = kAttnTile * D, kStage = 2 * kTile, NT = kRowsNT;
  constexpr int kHalf = 2 * 128 * D;         // query operand of a half: hi rows, then lo rows
  constexpr int kWide = kAttnTile * D * 2;   // widened value tile: D / 64 blocks of 128 tokens x 64 elements
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  RowsCtl<D>& c = *reinterpret_cast<RowsCtl<D>*>(smem_raw + (base - raw));
  const uint32_t ring = base + rows_ctl_bytes<D>(), qbuf = ring + S * kStage, wide = qbuf + 2 * kHalf;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &c.abort;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&c.kfull[i]), 1);
      mbar_init(smem_u32(&c.vfull[i]), 1);
      mbar_init(smem_u32(&c.empty[i]), 5);  // the last score product, the widening warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&c.sfull[i]), 2);  // the product, and the thread that saw the page scales
      mbar_init(smem_u32(&c.pfull[i]), 8);
      mbar_init(smem_u32(&c.pvdone[i]), 1);
      mbar_init(smem_u32(&c.wfull[i]), 4);
      mbar_init(smem_u32(&c.wempty[i]), 1);
      mbar_init(smem_u32(&c.qfull[i]), 8);
    }
    mbar_init(smem_u32(&c.drain), 1);
    for (int i = 0; i < kAttnQueue; ++i) {
      mbar_init(smem_u32(&c.segfull[i]), 1);
      mbar_init(smem_u32(&c.segempty[i]), 17);  // the softmax warps and the MMA thread
    }
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == 21) {
    tmem_alloc(smem_u32(&c.tmem), 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;  // scores (and weights) of the halves, then their outputs, 128 columns each
  // (only now: a dependent that allocates tensor memory must not come first)
  pdl_launch_dependents();
  pdl_wait();

  // After a wait that ran out (abort) the waits of warps that meet at barriers
  // fall through, so that they keep meeting until the segments end.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait_or_abort(smem_u32(bar), parity, abort_flag)) {
      if (!*abort_flag) report_error(p.err, kErrWaitMma);
      *abort_flag = 1;
    }
    __syncwarp();
  };

  if (warp == 20) {
    attn_walk<D, NT>(c, p, tmK, tmV, ring);
  } else if (warp == 21) {
    // ------------------------------------------------------------- MMA issuer
    // Order: PV of half 0, next scores of half 0, PV of half 1, next scores of
    // half 1: the weights of one half are computed under the other's products.
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_e4m3_f32(128, kAttnTile);
      constexpr uint32_t idesc_o = idesc_f16_f32(128, D) | (1u << 16);  // V is N-major
      bool ok = true;
      auto need = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !mbar_wait_or_abort(smem_u32(bar), parity, abort_flag)) {
          if (!*abort_flag) report_error(p.err, kErrWaitFull);
          *abort_flag = 1;
          ok = false;
        }
        return ok;
      };
      int sq = 0, i = 0;         // segments, tiles of the CTA
      int done[2] = {0, 0};      // tiles of each half whose weights were used
      int filled[2] = {0, 0};    // its query operands
      while (ok) {
        const int qi = sq % kAttnQueue;
        if (!need(&c.segfull[qi], (sq / kAttnQueue) & 1)) break;
        const int kind = c.seg[qi].kind, n = c.seg[qi].tb - c.seg[qi].ta, halves = c.seg[qi].nrows > 128 ? 2 : 1;
        mbar_arrive(smem_u32(&c.segempty[qi]));
        if (kind & kSegStop) break;
        ++sq;
        for (int k = 0; k <= n && ok; ++k) {
          const int x = i + k, y = x - 1;  // tile to score, tile to weigh
          for (int j = 0; j < halves && ok; ++j) {
            const uint32_t s_cols = tmem + (uint32_t)(j * 128), o_cols = tmem + (uint32_t)(256 + j * 128);
            if (k > 0) {
              if (!need(&c.wfull[y & 1], (y >> 1) & 1) || !need(&c.pfull[j], done[j] & 1)) break;
              tc_fence_after();
              const uint64_t wd = smem_desc_rows<128>(wide + (uint32_t)(y & 1) * kWide, kAttnTile * 128);
#pragma unroll
              for (int kk = 0; kk < kAttnTile / 16; ++kk)
                mma_bf16_tmem_a(o_cols, s_cols + (uint32_t)(kk * 8 + (kk < 4 ? 0 : 32)), wd + (uint64_t)(kk * (16 * 128 >> 4)), idesc_o,
                                (k > 1 || kk > 0) ? 1u : 0u);
              mma_commit(smem_u32(&c.pvdone[j]));
              if (j == halves - 1) mma_commit(smem_u32(&c.wempty[y & 1]));
              ++done[j];
            }
            if (k < n) {
              if (k == 0 && !need(&c.qfull[j], filled[j]++ & 1)) break;
              if (!need(&c.kfull[x % S], (x / S) & 1)) break;
              if (k > 0 && !need(&c.pvdone[j], (done[j] - 1) & 1)) break;  // the weights lie where the scores go
              tc_fence_after();
              const uint64_t kd = smem_desc_rows<D>(ring + (uint32_t)(x % S) * kStage + kTile);
              const uint64_t qd = smem_desc_rows<D>(qbuf + (uint32_t)(j * kHalf));
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) mma_e4m3(s_cols, qd + (uint64_t)(kk * 2), kd + (uint64_t)(kk * 2), idesc_s, kk > 0);
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_e4m3(s_cols, qd + (uint64_t)((128 * D >> 4) + kk * 2), kd + (uint64_t)(kk * 2), idesc_s, 1u);
              mma_commit(smem_u32(&c.sfull[j]));
              mbar_arrive(smem_u32(&c.sfull[j]));
              if (j == halves - 1) mma_commit(smem_u32(&c.empty[x % S]));
            }
          }
        }
        i += n;
      }
      mma_commit(smem_u32(&c.drain));
      if (!mbar_wait(smem_u32(&c.drain), 0)) report_error(p.err, kErrDrain);
    }
  } else if (warp >= 16) {
    // --------------------------------------------------------------- widen V
    // Thread = token: its D codes to FP16, zeros where no row sees it (0 x NaN
    // must not reach the product).  In tiles whose rows see different tokens a
    // NaN becomes zero too, and the softmax threads are told.
    const int tok = tid - 512;
    for (int i = 0;; ++i) {
      const int slot = i % S, meta = i % M, buf = i & 1;
      wait(&c.vfull[slot], (i / S) & 1);
      wait(&c.kfull[slot], (i / S) & 1);  // (orders the reads of what is written beside the copies)
      if (*abort_flag || (c.flags[meta] & 8)) break;
      wait(&c.wempty[buf], ((i >> 1) & 1) ^ 1);
      const int flags = c.flags[meta];
      const bool live = !flags || (tok >= c.live[meta][0] && tok < c.live[meta][1] &&
                                   c.vexp[meta][tok >> p.cache.page_shift] > -INFINITY);
      const uint32_t vt = ring + (uint32_t)slot * kStage, wt = wide + (uint32_t)buf * kWide;
      bool nans = false;
      if (flags & 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c.nan_mask[buf][tok][e] = 0u;
      }
#pragma unroll 2
      for (int k = 0; k < D / 16; ++k) {
        uint4 u = lds128(vt + swizzled<D>(tok, k));
        if (!live) u = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
        uint32_t h[8];
        uint32_t nan = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[2 * e] = widen2<0x9180>(w4[e]);
          h[2 * e + 1] = widen2<0xB3A2>(w4[e]);
          nan |= (w4[e] & 0x7F7F7F7Fu) + 0x01010101u;
        }
        if (__builtin_expect(nan & 0x80808080u, 0)) {
          uint32_t mask = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if ((w4[e >> 2] >> (8 * (e & 3)) & 0x7F) == 0x7F) {
              const uint32_t at = (e & 1) ? 0xFFFF0000u : 0x0000FFFFu;
              h[e >> 1] = (flags & 2) ? h[e >> 1] & ~at : h[e >> 1] | (at & 0x7FFF7FFFu);
              mask |= 1u << e;
            }
          if (flags & 2) c.nan_mask[buf][tok][k >> 1] |= mask << ((k & 1) * 16);
          nans = true;
        }
        // 16 elements: two chunks of the token's row in block k / 4
        const uint32_t at = wt + (uint32_t)(k / 4) * (kAttnTile * 128);
        sts128(at + swizzled<128>(tok, (k & 3) * 2), h[0], h[1], h[2], h[3]);
        sts128(at + swizzled<128>(tok, (k & 3) * 2 + 1), h[4], h[5], h[6], h[7]);
      }
      if (flags & 2) {
        const unsigned any = __ballot_sync(0xffffffffu, nans);
        if (lane == 0) c.nan_tokens[buf][warp - 16] = any;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&c.wfull[buf]));
        mbar_arrive(smem_u32(&c.empty[slot]));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int half = warp >> 3, sub = warp >> 2 & 1, row = tid & 127, ht = tid & 255;
    auto meet = [&] {  // the half's 8 warps
      __syncwarp();
      named_bar_sync(1 + half, 256);
    };
    const int pair_bar = 3 + half * 4 + (warp & 3);  // the two warps of a row
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // tensor-memory lanes of this warp
    const uint32_t s_cols = tmem + lanes + (uint32_t)(half * 128), o_cols = tmem + lanes + (uint32_t)(256 + half * 128);
    int i = 0, mine = 0, sq = 0;  // tiles of the CTA, tiles of this half, segments
    while (true) {
      const int qi = sq % kAttnQueue;
      if (ht == 0) c.go[half][sq & 1] = mbar_wait_or_abort(smem_u32(&c.segfull[qi]), (sq / kAttnQueue) & 1, abort_flag) ? 1 : 0;
      meet();
      if (!c.go[half][sq & 1]) {
        if (ht == 0 && !*abort_flag) report_error(p.err, kErrWaitFull);
        *abort_flag = 1;
        break;
      }
      const AttnSeg g = c.seg[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.segempty[qi]));
      ++sq;
      if (g.kind & kSegStop) break;
      if (g.nrows <= 128 * half) {  // no rows of this half
        i += g.tb - g.ta;
        continue;
      }
      // ------------------------------------------------------- query operand
      // D / 8 lanes a row, D / 16 passes, two rows of a thread under way.
      {
        constexpr int kLanes = D / 8, kRows = 256 / kLanes;
        const int l = ht % kLanes;
        auto load_row = [&](int pass) {
          const int q = 128 * half + pass * kRows + ht / kLanes;
          if (q >= g.nrows) return make_uint4(0u, 0u, 0u, 0u);
          const int r = g.r0 + q, tok = div_group(p, r), head = g.h * p.group + r - tok * p.group;
          return *reinterpret_cast<const uint4*>(p.q.p + (long long)(g.row0 + tok) * p.q.ts + (long long)head * p.q.hs + 8 * l);
        };
        uint4 v0 = load_row(0), v1 = load_row(1);
#pragma unroll 1
        for (int pass = 0; pass < kLanes / 2; ++pass) {
          const uint4 v = v0;
          v0 = v1;
          if (pass + 2 < kLanes / 2) v1 = load_row(pass + 2);
          const int q = pass * kRows + ht / kLanes;
          // (a negative scale turns the queries' signs: the factor is positive)
          const QuerySplit s = split_query<kLanes>(v, p.scale_log2 < 0.f ? -1.f : 1.f, 1.f);
          const uint32_t at = qbuf + (uint32_t)(half * kHalf + (l & 1) * 8) + swizzled<D>(q, l >> 1);
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(s.hi.x), "r"(s.hi.y) : "memory");
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + 128 * D), "r"(s.lo.x), "r"(s.lo.y) : "memory");
          if (l == 0) c.qf[128 * half + q] = s.factor * fabsf(p.scale_log2);
        }
        fence_proxy_async_smem();
        meet();  // (the factors, too)
        if (lane == 0) mbar_arrive(smem_u32(&c.qfull[half]));
      }
      const int q = 128 * half + row, r = g.r0 + q, rtok = div_group(p, r);
      const bool real = q < g.nrows;
      const int last = real ? row_last(g.first, rtok) : -1;
      const int see0 = row_first(g.tlo, last, p.window), see1 = min(g.thi - 1, last);
      // (a padding row's scores are all -inf: its query, NaN perhaps, has no part in them)
      const float qf = see0 <= see1 ? c.qf[q] : 0.f;
      // Factor of a page's scores: with the key scale it may underflow (a row of
      // zeros has qf near 2^-129, a page of zeros the scale 2^-64), and a masked
      // score, -inf, times zero is not -inf.  A score is below 2^24 in magnitude,
      // so what is below 2^-100 multiplies it to nothing all the same.
      auto score_factor = [&](float ks) {
        const float f = ks * qf;
        return f < 0x1p-100f ? 0x1p-100f : f;  // (a NaN stays)
      };
      float R = 0.f, l = 0.f;
      bool unset = true;  // whether the row has seen no position yet: R is its first maximum
      unsigned nan_d[4] = {0u, 0u, 0u, 0u};  // elements of the output that saw a NaN value
      for (int t = g.ta; t < g.tb; ++t, ++i, ++mine) {
        const int meta = i % M;
        wait(&c.sfull[half], mine & 1);
        tc_fence_after();
        const int flags = c.flags[meta], ps = p.cache.page_shift;
        const int c0 = see0 - t * kAttnTile, cn = see1 - t * kAttnTile - c0;  // columns that the row sees: c0 .. c0 + cn
        // The loops over a thread's columns stay rolled: unrolled, the body
        // does not fit the instruction caches, and the warps of four roles
        // then wait for instructions most of the time (a chunk of a prompt:
        // 236 us unrolled, 129 rolled, both with one thread a row).
        uint32_t x[32];
        if (__builtin_expect(flags, 0)) {  // what the row does not see: no score
#pragma unroll 1
          for (int k = 2 * sub; k < 2 * sub + 2; ++k) {
            tmem_ld32(s_cols + 32 * k, x);
            tmem_wait_ld32(x);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bool there = cn >= 0 && c.vexp[meta][(32 * k + 16 * h) >> ps] > -INFINITY;
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                w[e] = there && (unsigned)(32 * k + 16 * h + e - c0) <= (unsigned)cn ? x[16 * h + e] : 0xFF800000u;
              tmem_st16(s_cols + 32 * k + 16 * h, w);
            }
          }
          tmem_wait_st();
        }
        float top = -INFINITY;
#pragma unroll 1
        for (int k = 2 * sub; k < 2 * sub + 2; ++k) {
          tmem_ld32(s_cols + 32 * k, x);
          tmem_wait_ld32(x);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int pi = (32 * k + 16 * h) >> ps;
            float m[2] = {__uint_as_float(x[16 * h]), __uint_as_float(x[16 * h + 1])};
#pragma unroll
            for (int e = 2; e < 16; ++e) m[e & 1] = fmaxf(m[e & 1], __uint_as_float(x[16 * h + e]));
            top = fmaxf(top, fmaf(fmaxf(m[0], m[1]), score_factor(c.kscale[meta][pi]), c.vexp[meta][pi]));
          }
        }
        if (named_bar_or(pair_bar, 64, top > (unset ? -3.0e38f : R + 7.5f))) {  // (weights are 256 p: FP16 ends below 2^16)
          c.pair[half][sub][row] = top;
          __syncwarp();
          named_bar_sync(pair_bar, 64);
          top = fmaxf(top, c.pair[half][sub ^ 1][row]);
          const bool move = top > (unset ? -3.0e38f : R + 7.5f);
          const float now = move ? ceilf(top) : R, a = move && !unset ? exp2_whole(R - now) : 1.f;
          unset = unset && !move;
          R = now;
          l *= a;
          if (t > g.ta) {  // (the product before is done: its weights' place has new scores)
#pragma unroll 1
            for (int n = 0; n < D / 32; ++n) {  // this thread's half of the accumulator
              const uint32_t at = o_cols + (uint32_t)(sub * (D / 2) + 16 * n);
              float y[16];
              uint32_t w[16];
              tmem_ld16(at, y);
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(y[e] * a);
              tmem_st16(at, w);
            }
          }
        }
        // Weights, 256 p in FP16, over the first 32 of the thread's columns: a
        // chunk's lie where scores were that are read already.
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          tmem_ld32(s_cols + 64 * sub + 32 * k, x);
          tmem_wait_ld32(x);
          uint32_t w[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int pi = (64 * sub + 32 * k + 16 * h) >> ps;
            const float ve = c.vexp[meta][pi], kq = score_factor(c.kscale[meta][pi]), add = (ve + 8.f) - R;
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float z0 = ex2(fmaf(__uint_as_float(x[16 * h + 2 * e]), kq, add));
              const float z1 = ex2(fmaf(__uint_as_float(x[16 * h + 2 * e + 1]), kq, add));
              sum[0] += z0, sum[1] += z1;
              w[8 * h + e] = pack_f16(z0, z1);
            }
            l = fmaf(sum[0] + sum[1], ve > -INFINITY ? kv_exp2i(-(int)ve) : 0.f, l);  // without the value scale
          }
          tmem_st16(s_cols + 64 * sub + 16 * k, w);
        }
        tmem_wait_st();
        if (__builtin_expect(flags & 2, 0)) {
          wait(&c.wfull[i & 1], (i >> 1) & 1);
          for (int m = 0; m < 4; ++m)
            for (unsigned left = c.nan_tokens[i & 1][m]; left; left &= left - 1) {
              const int k = 32 * m + __ffs(left) - 1;
              if (cn < 0 || (unsigned)(k - c0) > (unsigned)cn) continue;
#pragma unroll
              for (int e = 0; e < 4; ++e) nan_d[e] |= c.nan_mask[i & 1][k][e];
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.pfull[half]));
      }
      // ------------------------------------------------------- the segment's end
      wait(&c.pvdone[half], (mine - 1) & 1);
      tc_fence_after();
      c.pair[half][sub][row] = l;
      meet();
      l = c.pair[half][0][row] + c.pair[half][1][row];
      const bool whole = (g.kind & (kSegStart | kSegEnd)) == (kSegStart | kSegEnd);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int head = g.h * p.group + r - rtok * p.group;
      __nv_bfloat16* out = p.out.p + (long long)(g.row0 + rtok) * p.out.ts + (long long)head * p.out.hs;
      float* part = p.part_o + ((long long)g.slot * NT + q) * D;
#pragma unroll 1
      for (int k = sub * (D / 64); k < (sub + 1) * (D / 64); ++k) {  // this thread's half of the row
        uint32_t x[32];
        tmem_ld32(o_cols + 32 * k, x);
        tmem_wait_ld32(x);
        const unsigned nan = k == 0 ? nan_d[0] : k == 1 ? nan_d[1] : k == 2 ? nan_d[2] : nan_d[3];
        if (__builtin_expect(nan != 0, 0)) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (nan >> e & 1) x[e] = 0x7fffffffu;
        }
        if (real && whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float z[8];
#pragma unroll
            for (int f = 0; f < 8; ++f) z[f] = __uint_as_float(x[8 * e + f]) * inv;
            *reinterpret_cast<uint4*>(out + 32 * k + 8 * e) =
                make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]), pack_bf16(z[6], z[7]));
          }
        } else if (real) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(part + 32 * k + 4 * e) = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
      }
      if (real && !whole && sub == 0) p.part_ml[(long long)g.slot * NT + q] = make_float2(unset ? -3.0e38f : R, l);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 21) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace sgr
