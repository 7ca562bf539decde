// sgr_kv_attn_few.cuh -- attention over the paged E4M3 cache for few query rows
// a key/value head (decode, verification of drafted tokens):
//
//     o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q.k_t)
//
// Per row tile (NT = 8, 16, 24 or 32 rows) and 128-token tile of the cache:
//
//     S^T [128 tokens, NT] = K Q^T      codes of K as they are in the cache
//     P^T = 2^(S' - R)                  one thread per token
//     O^T [D, NT]          = V^T P^T    codes of V as they are, read M-major
//
// Both products run on the FP8 tensor core (tcgen05.mma kind::f8f6f4) with
// the cache's codes as the 128-row operand straight from TMA, so that nothing
// is converted per cached element.  The small operands are brought into E4M3
// in parts, each the code of 32 times what the one before left.  Queries, each
// row scaled by a power of two that puts its largest magnitude in [128, 256),
// have two, b = hi + lo / 32: 8 significant bits (all of a BF16 query) down to
// 2^-14 of the largest and an absolute 2^-22 of it below.  Weights have three,
// b = w0 + w1 / 32 + w2 / 1024, off by at most 2^-11 of the weight (half of it
// from FP16 on the way) down to b = 2^-8 and by 2^-20, half a step, below.  The
// parts' rows sit side by side in the operand (2 NT or 3 NT columns of the
// accumulator) and are added in FP32.
//
// Softmax: weights are 2^(s' - R) with a whole number R for each column that
// only moves, up, when a score exceeds it (one vote of the four warps a tile;
// then the tile's maxima are found), so what came before is rescaled seldom
// and by a power of two: exactly.  The product of a tile is read back and
// accumulated in registers (thread d holds o[.][d]); no accumulator in tensor
// memory is ever rescaled.  A page's key scale multiplies the score; its value
// scale 2^e is added to the exponent of P and taken out of the sum of weights
// again, so a weight is p times its page's value scale.  The largest is at 2^6
// or above once R has moved: a weight is good to 2^-11 down to 2^-14 of the
// largest and to 2^-26 of the largest below, and n weights far below it are
// off by n 2^-26 of it together at most, less than BF16's rounding up to some
// 2^17 positions.  (Two parts leave 2^-21: of 131071 equal weights 2^-20
// of the largest, an eighth of the sum, a third was lost.)
//
// Bound: the cache bytes, 2 D a token and key/value head, each read once per
// row tile, where there are enough of them: 96 sequences of up to 16384 (64
// heads over 8, 1.63 GB) 240 us, 6.8 TB/s, a plain copy's rate; one of 200003
// (410 MB) 70 us.  With fewer bytes the CTAs' beginning (5 us: launch, tensor
// memory, first page, first run of the code) and the join (3 us): 32 sequences
// of up to 4096 (28 heads over 4, 60.6 MB) 19.4 us, one of 333 8.2 us.  With
// more rows a head the softmax: 20 rows (D = 64, 38.7 MB) 29 us, issue slots
// 61% taken.  (Of which the weights' third part 0.4 us with 8 rows, 2 with 20.)
//
// Roles: a group of 4 softmax warps for every 8 rows (thread = token, then =
// element d), one warp that walks the work, loads pages by TMA and hands out
// segments, one that issues the MMAs, two that bring the next segments'
// queries into the operand.  Two CTAs an SM, so that one computes while the
// other waits (one with 32 rows, whose registers and shared memory two would
// not fit; three with 8 rows were slower).
#pragma once

#include "sgr_kv_attn.cuh"

namespace sgr {

// Error word, beside the codes of sgr_ptx.cuh: a CTA's shared memory does not
// begin where the kernel needs it.
constexpr unsigned kErrSmemAlign = 8;

template <int D, int NT>
struct AttnShape {
  static constexpr int kC = 8;             // columns a softmax thread
  static constexpr int kGroups = NT / kC;  // of 4 softmax warps
  static constexpr int kSoftmax = 4 * kGroups;
  static constexpr int kThreads = 32 * (kSoftmax + 4);
  static constexpr int kCtas = NT > 24 ? 1 : 2;  // an SM
  static constexpr int kCols = 2 * NT;                     // the queries' two parts
  static constexpr int kWCols = (3 * NT + 15) / 16 * 16;  // the weights' three (the product's width is a multiple of 16)
  static constexpr int kTileBytes = kAttnTile * D;
  static constexpr int kStageBytes = 2 * kTileBytes;  // V, then K
  // As many stages and query buffers as kCtas an SM allow.
  static constexpr int kStages = D == 128 ? (NT == 32 ? 5 : NT == 24 ? 2 : 3) : (NT == 32 ? 8 : NT == 8 ? 6 : 5);
  static constexpr int kQBufs = D == 128 && NT == 16 ? 2 : D == 128 && NT == 32 ? 3 : D == 64 && NT == 24 ? 2 : 4;
  static constexpr int kPBytes = kWCols * kAttnTile;
  static constexpr int kQBytes = kCols * D;
  static constexpr int kTmemCols = NT == 8 ? 128 : NT < 32 ? 256 : 512;  // S and O, two each (a power of two)
  static_assert(kTmemCols >= 2 * (kCols + kWCols), "two accumulators of each product");
};

template <int D, int NT>
struct AttnCtl {
  using Sh = AttnShape<D, NT>;
  static constexpr bool kStopStage = false;
  static constexpr int kStages = Sh::kStages, kMeta = kStages, S = kStages, Q = Sh::kQBufs, C = Sh::kC;
  uint64_t kfull[S], vfull[S], empty[S];
  uint64_t sfull[2], sempty[2], ofull[2], oempty[2], qfull[Q], qempty[Q], pfull, drain;
  uint64_t segfull[kAttnQueue], segempty[kAttnQueue];
  uint32_t tmem;
  int abort;
  int go[Sh::kGroups][2];
  unsigned nan_tokens[4];
  AttnSeg seg[kAttnQueue];
  float kscale[S][8], vexp[S][8];  // of a stage's pages
  int flags[S], live[S][2];        // flags: 1: some token is not live, 2: rows see different tokens; live tokens
  long long qout[Q][NT];           // a row's place in the output
  alignas(16) float qf[Q][NT];     // its score factor
  int qpos[Q][NT];                 // the last position that it sees
  alignas(16) float wmax[Sh::kSoftmax][C], wsum[Sh::kSoftmax][C];
  alignas(16) float ref[Sh::kSoftmax][C], alpha[Sh::kSoftmax][2][C];  // a warp's own copies
};

template <int D, int NT>
constexpr int attn_ctl_bytes() {
  return (int)((sizeof(AttnCtl<D, NT>) + 1023) / 1024 * 1024);
}

template <int D, int NT>
constexpr int attn_smem_bytes() {
  using S = AttnShape<D, NT>;
  return attn_ctl_bytes<D, NT>() + S::kStages * S::kStageBytes + S::kPBytes + S::kQBufs * S::kQBytes;
}

// Sums of C columns over the warp's lanes: lane l returns column l / (32 / C).
template <int C>
__device__ __forceinline__ float warp_column_sums(float (&x)[C]) {
  const int lane = threadIdx.x & 31;
  int d = 16;
#pragma unroll
  for (int n = C / 2; n > 0; n >>= 1, d >>= 1) {
    const bool upper = (lane & d) != 0;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float give = upper ? x[k] : x[k + n], keep = upper ? x[k + n] : x[k];
      x[k] = keep + __shfl_xor_sync(0xffffffffu, give, d);
    }
  }
#pragma unroll
  for (; d > 0; d >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], d);
  return x[0];
}

constexpr float kLoScale = 1.f / 32.f;

// Two values in [0, 256] -> their codes in three parts, one pair of bytes each:
// b = w0 + w1 / 32 + w2 / 1024.  (FP16 holds b to 11 bits, the rests exactly.)
__device__ __forceinline__ void split3(float a, float b, uint32_t& w01, uint32_t& w2) {
  asm("{\n\t.reg .b16 h, l, m;\n\t.reg .b32 x, y;\n\t"
      "cvt.rn.f16x2.f32 x, %3, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 h, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, h;\n\t"
      "sub.rn.f16x2 x, x, y;\n\t"
      "mul.rn.f16x2 x, x, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 l, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, l;\n\t"
      "sub.rn.f16x2 x, x, y;\n\t"
      "mul.rn.f16x2 x, x, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 m, x;\n\t"
      "mov.b32 %0, {h, l};\n\t"
      "mov.b32 %1, {m, m};\n\t}"
      : "=r"(w01), "=r"(w2)
      : "f"(a), "f"(b), "r"(0x50005000u));  // 0x5000 = 32
}

// x[q] = hi[q] + lo[q] / 32 of C accumulator columns at `hi`, the lo ones
// `apart` columns on.
template <int C>
__device__ __forceinline__ void tmem_ld_sum(uint32_t hi, uint32_t apart, float (&x)[C]) {
  static_assert(C == 8, "the load of two runs of 8 columns");
  float v[8], w[8];
  tmem_ld8x2(hi, hi + apart, v, w);
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] = fmaf(w[q], kLoScale, v[q]);
}

// Three runs of 8 consecutive columns of the same lanes.
__device__ __forceinline__ void tmem_ld8x3(uint32_t ta, uint32_t tb, uint32_t tc, float (&v)[8], float (&w)[8], float (&x)[8]) {
  uint32_t r[24];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(ta)
               : "memory");
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(tb)
               : "memory");
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23])
               : "r"(tc)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23])
               :
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = __uint_as_float(r[i]);
    w[i] = __uint_as_float(r[8 + i]);
    x[i] = __uint_as_float(r[16 + i]);
  }
}

// The same of three parts, w0 + w1 / 32 + w2 / 1024.
template <int C>
__device__ __forceinline__ void tmem_ld_sum3(uint32_t w0, uint32_t apart, float (&x)[C]) {
  static_assert(C == 8, "the load of three runs of 8 columns");
  float v[8], w[8];
  tmem_ld8x3(w0, w0 + apart, w0 + 2 * apart, x, v, w);
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] = fmaf(fmaf(w[q], kLoScale, v[q]), kLoScale, x[q]);
}

template <int D, int NT>
__global__ void __launch_bounds__(AttnShape<D, NT>::kThreads, AttnShape<D, NT>::kCtas)
    kv_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
  using Sh = AttnShape<D, NT>;
  constexpr int S = Sh::kStages, Q = Sh::kQBufs, C = Sh::kC, kCols = Sh::kCols, kWCols = Sh::kWCols, kSoftmax = Sh::kSoftmax;
  // (aligned by its declaration: room to align it by hand would cost 16-row
  // tiles of D = 128 their second CTA an SM)
  extern __shared__ __align__(1024) unsigned char attn_smem[];
  const uint32_t base = smem_u32(attn_smem);
  if (base & 1023u) {  // swizzled operands could not be read
    pdl_wait();
    if (threadIdx.x == 0) {
      report_error(p.err, kErrSmemAlign);
      p.pieces[blockIdx.x] = AttnPiece{};  // (nothing to join)
    }
    return;
  }
  AttnCtl<D, NT>& c = *reinterpret_cast<AttnCtl<D, NT>*>(attn_smem);
  const uint32_t ring = base + attn_ctl_bytes<D, NT>();
  const uint32_t pbuf = ring + S * Sh::kStageBytes, qbuf = pbuf + Sh::kPBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &c.abort;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&c.kfull[i]), 1);
      mbar_init(smem_u32(&c.vfull[i]), 1);
      mbar_init(smem_u32(&c.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&c.sfull[i]), 2);  // the product, and the thread that saw the page scales
      mbar_init(smem_u32(&c.sempty[i]), kSoftmax);
      mbar_init(smem_u32(&c.ofull[i]), 1);
      mbar_init(smem_u32(&c.oempty[i]), kSoftmax);
    }
    for (int i = 0; i < Q; ++i) {
      mbar_init(smem_u32(&c.qfull[i]), 2);
      mbar_init(smem_u32(&c.qempty[i]), 1 + kSoftmax);  // the last MMA that reads it, the softmax warps
    }
    mbar_init(smem_u32(&c.pfull), kSoftmax);
    mbar_init(smem_u32(&c.drain), 1);
    for (int i = 0; i < kAttnQueue; ++i) {
      mbar_init(smem_u32(&c.segfull[i]), 1);
      mbar_init(smem_u32(&c.segempty[i]), kSoftmax + 3);  // and the MMA and query warps
    }
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == kSoftmax + 1) {
    tmem_alloc(smem_u32(&c.tmem), Sh::kTmemCols);
    tmem_relinquish();
  }
  if (tid == 32) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  // (only now: a dependent that allocates tensor memory must not come first)
  pdl_launch_dependents();
  if (warp < kSoftmax + 2) pdl_wait();  // (the query warps do after their dry run)

  if (warp == kSoftmax) {
    attn_walk<D, NT>(c, p, tmK, tmV, ring);
  } else if (warp == kSoftmax + 1) {
    // ------------------------------------------------------------- MMA issuer
    // Issues whichever of the two products can go: V^T P^T of the oldest tile
    // whose weights are written, or K Q^T of the next one.  Neither waits for
    // the other's inputs.
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_e4m3_f32(kAttnTile, kCols), idesc_o = idesc_e4m3_f32(kAttnTile, kWCols) | (1u << 15);
      const uint32_t acc_o = tmem + 2 * kCols;
      int sq = 0, filled = -1, t = 0, t_end = 0;  // segments read, query buffer in use, its tiles
      int i = 0, islot = 0, k = 0, kslot = 0;     // tiles scored, tiles weighted
      uint32_t ipar = 0, kpar = 0;
      bool fresh = false, stop = false, ok = true;
      uint64_t since = 0;
      unsigned idle = 0;
      while (ok && (!stop || k < i)) {
        if (k < i && mbar_test_wait(smem_u32(&c.pfull), k & 1) && mbar_test_wait(smem_u32(&c.vfull[kslot]), kpar) &&
            mbar_test_wait(smem_u32(&c.oempty[k & 1]), ((k >> 1) & 1) ^ 1)) {
          tc_fence_after();
          // D = 64: the upper half of the 128 rows reads the K tile behind V;
          // its rows of the accumulator are not used.
          const uint64_t vd = smem_desc_rows<D>(ring + (uint32_t)kslot * Sh::kStageBytes, Sh::kTileBytes);
          const uint64_t pd = smem_desc_rows<128>(pbuf);
#pragma unroll
          for (int kk = 0; kk < kAttnTile / 32; ++kk)
            mma_e4m3(acc_o + (k & 1) * kWCols, vd + (uint64_t)(kk * (32 * D >> 4)), pd + (uint64_t)(kk * 2), idesc_o, kk > 0);
          mma_commit(smem_u32(&c.ofull[k & 1]));
          mma_commit(smem_u32(&c.empty[kslot]));
          ++k;
          if (++kslot == S) {
            kslot = 0;
            kpar ^= 1u;
          }
          idle = 0;
          continue;
        }
        if (!stop && t == t_end) {
          const int qi = sq % kAttnQueue;
          if (mbar_test_wait(smem_u32(&c.segfull[qi]), (sq / kAttnQueue) & 1)) {
            stop = (c.seg[qi].kind & kSegStop) != 0;
            t = c.seg[qi].ta;
            t_end = c.seg[qi].tb;
            mbar_arrive(smem_u32(&c.segempty[qi]));
            ++sq;
            ++filled;
            fresh = true;
            idle = 0;
            continue;
          }
        } else if (!stop && (!fresh || mbar_test_wait(smem_u32(&c.qfull[filled % Q]), (filled / Q) & 1)) &&
                   mbar_test_wait(smem_u32(&c.kfull[islot]), ipar) &&
                   mbar_test_wait(smem_u32(&c.sempty[i & 1]), ((i >> 1) & 1) ^ 1)) {
          fresh = false;
          tc_fence_after();
          const uint64_t kd = smem_desc_rows<D>(ring + (uint32_t)islot * Sh::kStageBytes + Sh::kTileBytes);
          const uint64_t qd = smem_desc_rows<D>(qbuf + (uint32_t)(filled % Q) * Sh::kQBytes);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_e4m3(tmem + (i & 1) * kCols, kd + (uint64_t)(kk * 2), qd + (uint64_t)(kk * 2), idesc_s, kk > 0);
          mma_commit(smem_u32(&c.sfull[i & 1]));
          mbar_arrive(smem_u32(&c.sfull[i & 1]));
          if (++t == t_end) mma_commit(smem_u32(&c.qempty[filled % Q]));
          ++i;
          if (++islot == S) {
            islot = 0;
            ipar ^= 1u;
          }
          idle = 0;
          continue;
        }
        // Nothing to issue: bounded, as every wait.
        if (idle == 0) since = globaltimer_ns();
        if ((++idle & 63u) == 0) {
          if (*abort_flag) ok = false;
          if (globaltimer_ns() - since > SGR_WAIT_LIMIT_NS) {
            report_error(p.err, kErrWaitFull);
            *abort_flag = 1;
            ok = false;
          }
        }
      }
      mma_commit(smem_u32(&c.drain));
      if (!mbar_wait(smem_u32(&c.drain), 0)) report_error(p.err, kErrDrain);
    }
  } else if (warp >= kSoftmax + 2) {
    // ----------------------------------------------------------- query operand
    // First a dry run over no rows: a CTA's first run of this code waits for
    // its instructions, on the way to the first scores (8.2 against 9.8 us for
    // one short sequence).  Dry runs of the other roles gained nothing.
    constexpr int kLanes = D / 8, kRows = 64 / kLanes, kPass = NT / kRows;
    const int qt = tid - 32 * (kSoftmax + 2), l = qt % kLanes;
    int sq = 0, buf = 0;
    uint32_t par = 0;
    bool dry = true;
    while (true) {
      const int qi = sq % kAttnQueue;
      bool ok = true;
      AttnSeg g{};
      if (!dry) {
        if (lane == 0) ok = mbar_wait_nap<kNap>(smem_u32(&c.segfull[qi]), (sq / kAttnQueue) & 1, abort_flag);
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        g = c.seg[qi];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.segempty[qi]));
        ++sq;
        if (g.kind & kSegStop) break;
      }
      // Row `pass` of this thread's: two are under way while one is converted.
      auto load_row = [&](int pass, long long& out_at, int& pos) {
        const int q = pass * kRows + qt / kLanes;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        pos = -1;  // a row that is none sees nothing
        out_at = 0;
        if (q < g.nrows) {
          const int r = g.r0 + q, tok = div_group(p, r), head = g.h * p.group + r - tok * p.group;
          pos = row_last(g.first, tok);
          out_at = (long long)(g.row0 + tok) * p.out.ts + (long long)head * p.out.hs;
          v = *reinterpret_cast<const uint4*>(p.q.p + (long long)(g.row0 + tok) * p.q.ts + (long long)head * p.q.hs + 8 * l);
        }
        return v;
      };
      long long out0, out1 = 0;
      int pos0, pos1 = -1;
      uint4 v0 = load_row(0, out0, pos0), v1 = v0;
      if (kPass > 1) v1 = load_row(1, out1, pos1);
      if (lane == 0 && !dry) ok = mbar_wait_nap<kNap>(smem_u32(&c.qempty[buf]), par ^ 1u, abort_flag);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
#pragma unroll 1
      for (int i = 0; i < kPass; ++i) {
        const int q = i * kRows + qt / kLanes, pos = pos0;
        const long long out_at = out0;
        const uint4 v = v0;
        v0 = v1, out0 = out1, pos0 = pos1;
        if (i + 2 < kPass) v1 = load_row(i + 2, out1, pos1);
        const QuerySplit s = split_query<kLanes>(v, 1.f, 32.f);
        const uint32_t qb = qbuf + (uint32_t)(buf * Sh::kQBytes) + (uint32_t)((l & 1) * 8);
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qb + swizzled<D>(q, l >> 1)), "r"(s.hi.x), "r"(s.hi.y) : "memory");
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qb + swizzled<D>(NT + q, l >> 1)), "r"(s.lo.x), "r"(s.lo.y) : "memory");
        if (l == 0) {
          c.qf[buf][q] = s.factor * p.scale_log2;
          c.qpos[buf][q] = pos;
          c.qout[buf][q] = out_at;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (dry) {
        dry = false;
        pdl_wait();
        continue;
      }
      if (lane == 0) mbar_arrive(smem_u32(&c.qfull[buf]));
      if (++buf == Q) {
        buf = 0;
        par ^= 1u;
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    // After a wait that ran out (abort) the waits fall through, so that the
    // warps keep meeting at their barriers until the segments end.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar_wait_or_abort(smem_u32(bar), parity, abort_flag)) {
        if (!*abort_flag) report_error(p.err, kErrWaitMma);
        *abort_flag = 1;
      }
      __syncwarp();
    };
    const int group = warp >> 2, tok = tid & 127, q0 = group * C;  // columns q0 .. q0 + C - 1
    auto meet = [&] {  // the group's 4 warps
      __syncwarp();
      named_bar_sync(1 + group, 128);
    };
    const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21) + (uint32_t)q0;  // tensor-memory lanes of this warp
    float o[C], l[C];
    float run = 0.f;  // R of column q0 + lane
    unsigned nan_rows = 0;
    int i = 0, slot = 0, sq = 0, buf = 0;
    uint32_t par = 0, qpar = 0;
    bool scaled_before = false;  // whether R moved with the tile before
    // O of tile k (after its wait), read back and accumulated.
    auto accumulate = [&](int k, bool scaled) {
      tc_fence_after();
      float x[C];
      tmem_ld_sum3<C>(lane_base + 2 * kCols + (k & 1) * kWCols, NT, x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.oempty[k & 1]));
      if (scaled) {
#pragma unroll
        for (int q = 0; q < C; ++q) o[q] *= c.alpha[warp][k & 1][q];
      }
#pragma unroll
      for (int q = 0; q < C; ++q) o[q] += x[q];
    };
    while (true) {
      const int qi = sq % kAttnQueue;
      if (tok == 0) c.go[group][sq & 1] = mbar_wait_or_abort(smem_u32(&c.segfull[qi]), (sq / kAttnQueue) & 1, abort_flag) ? 1 : 0;
      meet();
      if (!c.go[group][sq & 1]) {
        if (tok == 0 && !*abort_flag) report_error(p.err, kErrWaitFull);
        *abort_flag = 1;
        break;
      }
      const AttnSeg g = c.seg[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.segempty[qi]));
      ++sq;
      if (g.kind & kSegStop) break;
      wait(&c.qfull[buf], qpar);
#pragma unroll
      for (int q = 0; q < C; ++q) o[q] = l[q] = 0.f;
      run = -3.0e38f;
      if (lane < C) c.ref[warp][lane] = run;
      nan_rows = 0;
      __syncwarp();
      for (int t = g.ta; t < g.tb; ++t) {
        const int sb = i & 1;
        wait(&c.sfull[sb], (i >> 1) & 1);
        tc_fence_after();
        float x[C];
        tmem_ld_sum<C>(lane_base + sb * kCols, NT, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.sempty[sb]));
        const int pi = tok >> p.cache.page_shift, flags = c.flags[slot], pos = t * kAttnTile + tok;
        const float ks = c.kscale[slot][pi], ve = c.vexp[slot][pi];
        const bool live = !(flags & 1) || (tok >= c.live[slot][0] && tok < c.live[slot][1] && ve > -INFINITY);
#pragma unroll
        for (int q = 0; q < C; ++q) x[q] = fmaf(x[q], ks * c.qf[buf][q0 + q], ve + 8.f);  // weights come as 256 p
        if (__builtin_expect(flags & 2, 0)) {
#pragma unroll
          for (int q = 0; q < C; ++q) {
            const int last = c.qpos[buf][q0 + q];
            if (!(live && row_sees(pos, last, p.window))) x[q] = -INFINITY;
          }
        } else if (!live) {
#pragma unroll
          for (int q = 0; q < C; ++q) x[q] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < C; ++q) top = fmaxf(top, x[q] - c.ref[warp][q]);
        const bool scaled = named_bar_or(1 + group, 128, top > 8.f);  // the most that the lower parts have room for: 32 times a rest of 8
        if (__builtin_expect(scaled, 0)) {
          // R of the columns that are exceeded moves one above the tile's
          // maximum (room for the next tiles); lane q keeps column q's.
          top = -INFINITY;
#pragma unroll
          for (int q = 0; q < C; ++q) {
            const float w = warp_max(x[q]);
            if (lane == q) top = w;
          }
          if (lane < C) c.wmax[warp][lane] = top;
          meet();
          if (lane < C) {
            const int w0 = warp & ~3;
            top = fmaxf(fmaxf(c.wmax[w0][lane], c.wmax[w0 + 1][lane]), fmaxf(c.wmax[w0 + 2][lane], c.wmax[w0 + 3][lane]));
            const float now = top - run > 8.f ? ceilf(top) - 7.f : run;
            c.alpha[warp][sb][lane] = exp2_whole(run - now);
            c.ref[warp][lane] = run = now;
          }
          __syncwarp();
#pragma unroll
          for (int q = 0; q < C; ++q) l[q] *= c.alpha[warp][sb][q];
        }
        const float iv = live ? kv_exp2i(-(int)ve) : 0.f;  // the value scale does not count in the sum of weights
#pragma unroll
        for (int q = 0; q < C; ++q) {
          x[q] = ex2(x[q] - c.ref[warp][q]);
          l[q] = fmaf(x[q], iv, l[q]);
        }
        const bool joined = t > g.ta;
        if (joined) wait(&c.ofull[(i - 1) & 1], ((i - 1) >> 1) & 1);  // the weights before are read
        if (__builtin_expect(flags, 0)) {
          wait(&c.vfull[slot], par);
          const uint32_t vt = ring + (uint32_t)slot * Sh::kStageBytes;
          // Values of tokens that no row sees must not reach the product
          // (0 x NaN): their codes become zeros.
          if (!live && group == 0) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + (uint32_t)(tok * D + k * 16)), "r"(0u) : "memory");
          }
          if (flags & 2) {
            // A NaN value that some rows see and others do not: those that do
            // get their NaN here, and the code becomes zero.
            bool nan = false;
            if (live && group == 0) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint4 u = lds128(vt + (uint32_t)(tok * D + k * 16));
                const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) nan |= (((w4[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
              }
            }
            const unsigned any = __ballot_sync(0xffffffffu, nan);
            if (lane == 0 && group == 0) c.nan_tokens[warp] = any;
            __syncwarp();
            named_bar_sync(1 + Sh::kGroups, 32 * kSoftmax);
            if ((c.nan_tokens[0] | c.nan_tokens[1] | c.nan_tokens[2] | c.nan_tokens[3]) != 0) {
              for (int k = 0; k < kAttnTile; ++k) {
                if (!(c.nan_tokens[k >> 5] >> (k & 31) & 1) || tok >= D) continue;
                if ((lds8(vt + swizzled<D>(k, tok >> 4) + (tok & 15)) & 0x7F) != 0x7F) continue;
                for (int q = 0; q < C; ++q) {
                  const int last = c.qpos[buf][q0 + q], kp = t * kAttnTile + k;
                  if (row_sees(kp, last, p.window)) nan_rows |= 1u << q;
                }
              }
              __syncwarp();
              named_bar_sync(1 + Sh::kGroups, 32 * kSoftmax);  // all have seen the codes
              if (nan) {
                for (int k = 0; k < D; ++k)
                  if ((lds8(vt + (uint32_t)(tok * D + k)) & 0x7F) == 0x7F) sts8(vt + (uint32_t)(tok * D + k), 0);
              }
            }
            __syncwarp();
          }
        }
        const uint32_t col = (uint32_t)(tok & 15), chunk = tok >> 4;
#pragma unroll
        for (int q = 0; q < C; q += 2) {
          uint32_t u, m;
          split3(x[q], x[q + 1], u, m);
          // (q0 and NT are multiples of 8: they do not change the swizzle)
          const uint32_t at0 = pbuf + q0 * 128 + swizzled<128>(q, chunk) + col, at1 = pbuf + q0 * 128 + swizzled<128>(q + 1, chunk) + col;
          sts8(at0, u);
          sts8(at1, u >> 8);
          sts8(at0 + NT * 128, u >> 16);
          sts8(at1 + NT * 128, u >> 24);
          sts8(at0 + 2 * NT * 128, m);
          sts8(at1 + 2 * NT * 128, m >> 8);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.pfull));
        if (joined) accumulate(i - 1, scaled_before);
        scaled_before = scaled;
        ++i;
        if (++slot == S) {
          slot = 0;
          par ^= 1u;
        }
      }
      wait(&c.ofull[(i - 1) & 1], ((i - 1) >> 1) & 1);
      accumulate(i - 1, scaled_before);
      // ------------------------------------------------------- the segment's end
      const float part = warp_column_sums<C>(l);
      if (lane % (32 / C) == 0) c.wsum[warp][lane / (32 / C)] = part;
      meet();
      const bool whole = (g.kind & (kSegStart | kSegEnd)) == (kSegStart | kSegEnd);
      if (lane < C) {
        const int w0 = warp & ~3;
        const float sum = c.wsum[w0][lane] + c.wsum[w0 + 1][lane] + c.wsum[w0 + 2][lane] + c.wsum[w0 + 3][lane];
        c.ref[warp][lane] = sum == 0.f ? 0.f : 1.f / sum;  // (R is not needed any more)
        if (!whole && (warp & 3) == 0 && q0 + lane < g.nrows)
          p.part_ml[(long long)g.slot * NT + q0 + lane] = make_float2(run, sum);
      }
      __syncwarp();
      if (tok < D) {
#pragma unroll
        for (int q = 0; q < C; ++q) {
          const float v = nan_rows >> q & 1 ? __int_as_float(0x7fffffff) : o[q];
          if (q0 + q < g.nrows) {
            if (whole)
              p.out.p[c.qout[buf][q0 + q] + tok] = __float2bfloat16(v * c.ref[warp][q]);
            else
              p.part_o[((long long)g.slot * NT + q0 + q) * D + tok] = v;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.qempty[buf]));
      if (++buf == Q) {
        buf = 0;
        qpar ^= 1u;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmax + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::kTmemCols);
  }
}

}  // namespace sgr
