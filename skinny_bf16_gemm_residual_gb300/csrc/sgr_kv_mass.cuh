// sgr_kv_mass.cuh -- the attention weight that cached positions get from the
// new tokens' rows, added to what they have (sgr_attention.h):
//
//     mass[t, h] += sum over rows r and heads of h's group of 2^(s_rt - L_r)
//     s = scale log2(e) q.k,   L = log2(e) lse
//
// With the rows' log-sum-exp known a position's sum needs its own key alone:
// one pass over K and no maxima.  As in the attention kernel
// (sgr_kv_attn_few.cuh) the codes of 128 keys are the 128-row operand of the FP8
// tensor core as they are,
//
//     S^T [128 keys, 2 rows] = K Q^T
//
// with the rows' queries in two E4M3 parts b = hi + lo / 32 side by side (8
// significant bits, all of a BF16 query, down to 2^-14 of its row's largest
// and an absolute 2^-22 of it below).  Thread = key: it reads its lane of the
// accumulator, adds the parts in FP32, and sums 2^(s - L) over the columns: in one
// thread for products of 8 or 16 rows, in two for larger ones, a half of the
// columns each, whose halves meet in shared memory once a tile.
//
// Bound: for few rows the keys' bytes, each read once (64 sequences of up to
// 16384, 64 heads of 128 over 8, 607 MB: 97 us, 6.3 TB/s); one request's of 333
// positions 5.4 us in a graph (launch, walk, first page).  For many rows a chain
// of product, its sums and the next product in each of two CTAs an SM, issue slots
// 55% taken (chunks of up to 500 tokens over 4001, 32 heads of 64 over 8, 87
// million weights: 59 us; the exponentials alone would take some 19).  In between
// 32 sequences of up to 8000 with 20 rows a head 42 us (32 heads of 128 over 8,
// 145 MB: 22 us at the copy peak), 8 of 5000 with 128 rows 35 (32 MB).  Registers
// bound the two-group kernels: 80 for two CTAs an SM, 16 bytes of spills with 32
// rows and 40 with 64.
//
// Rows that share a key/value head go in products of up to 64.  Up to 128 of
// them, their queries all in shared memory, meet a tile of keys while it is
// there (it is read once); more are several row tiles, whose sums go to the
// workspace and are added in order by a second kernel.  A sequence adds once to
// each of its positions: the same bits on every run, but for positions of pages
// that several sequences share, whose sums are added in any order.  Every CTA
// takes the same number of (row tile, key tile) units (attn_walk).
//
// Roles: four warps weigh (thread = key; eight for products of 32 rows or more,
// half of the columns each), one walks the work and loads pages, one issues the
// MMAs, two bring queries into the operand, a ring of products' worth of
// rows.
#pragma once

#include <climits>
#include <type_traits>

#include "sgr_kv_attn_few.cuh"
#include "sgr_kv_attn_rows.cuh"

namespace sgr {

struct MassParams {
  AttnParams a;  // (lse: input; out, partial sums and pieces unused)
  float* mass;
  long long page_stride, head_stride;  // elements
  float* part;  // [row tile][key/value head][128 tiles positions], NULL: one row tile a sequence
  int tiles;    // of a sequence, at most
  int max_new;  // rows of a sequence, at most
};

constexpr int kMassRows = 128;  // of the largest row tile

template <int D, int NT>
struct MassShape {
  static constexpr int kRows = NT < 64 ? NT : 64;  // of a product
  static constexpr int kCols = 2 * kRows;
  static constexpr int kAcc = kRows == 64 ? 2 : 4;  // accumulators
  static constexpr int kGroups = kRows >= 32 ? 2 : 1;  // of 4 weighing warps, each a part of a product's columns
  static constexpr int kWeigh = 4 * kGroups, kQuery = 2;  // warps
  static constexpr int kThreads = 32 * (kWeigh + 2 + kQuery);
  static constexpr int kTileBytes = kAttnTile * D;
  static constexpr int kSlotBytes = kCols * D;
  // As many stages of keys and slots of queries as two CTAs an SM allow.
  static constexpr int kStages = D == 128 ? (NT <= 16 ? 6 : NT == 32 ? 5 : 2) : (NT <= 16 ? 10 : NT == 32 ? 8 : 5);
  static constexpr int kSlots = NT == 16 || NT == 32 ? 3 : 4;
  static constexpr int kTmemCols = kAcc * kCols;
};

template <int D, int NT>
struct MassCtl {
  using Sh = MassShape<D, NT>;
  static constexpr bool kStopStage = false, kValues = false;
  static constexpr int kStages = Sh::kStages, kMeta = kStages, S = kStages, Q = Sh::kSlots;
  uint64_t kfull[S], empty[S];
  uint64_t sfull[Sh::kAcc], sempty[Sh::kAcc], qfull[Q], qempty[Q], drain;
  uint64_t segfull[kAttnQueue], segempty[kAttnQueue];
  uint32_t tmem;
  int abort;
  int go[2];
  AttnSeg seg[kAttnQueue];
  float kscale[S][8];  // of a stage's pages
  int page[S][8];      // (-1: not there)
  int flags[S], live[S][2];
  float sum[Sh::kGroups > 1 ? 2 : 1][kAttnTile];  // of the second group, two tiles
  alignas(16) float qf[Q][Sh::kRows];  // a row's score factor
  alignas(16) float ql[Q][Sh::kRows];  // and -L (-inf: a row that counts for nothing)
  int qpos[Q][Sh::kRows];              // the last position that it sees, by itself
  int qrow[Q][Sh::kRows];              // the row (of a tree's bits)
};

template <int D, int NT>
constexpr int mass_ctl_bytes() {
  return (int)((sizeof(MassCtl<D, NT>) + 1023) / 1024 * 1024);
}

template <int D, int NT>
constexpr int mass_smem_bytes() {
  using S = MassShape<D, NT>;
  return mass_ctl_bytes<D, NT>() + S::kStages * S::kTileBytes + S::kSlots * S::kSlotBytes;
}

// Where a row tile's sums of a key/value head go in `part`: a sequence's row
// tiles are numbered from one for every NT rows before it and one a sequence.
template <int NT>
__device__ __forceinline__ long long mass_part(const MassParams& p, int b, int row0, int j, int h) {
  const long long tile = (long long)row0 * p.a.group / NT + b + j;
  return (tile * p.a.cache.heads + h) * p.tiles * kAttnTile;
}

// hi and lo parts of C accumulator columns, the lo ones `apart` columns on.
template <int C>
__device__ __forceinline__ void tmem_ld_parts(uint32_t hi_at, uint32_t apart, float (&hi)[C], float (&lo)[C]) {
  static_assert(C == 8 || C == 16, "one load of each part");
  if constexpr (C == 8) {
    tmem_ld8x2(hi_at, hi_at + apart, hi, lo);
  } else {
    uint32_t r[32];
#define SGR_LD16(AT, O)                                                                                               \
  asm volatile(                                                                                                       \
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "                                                                       \
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"                                \
      : "=r"(r[O]), "=r"(r[O + 1]), "=r"(r[O + 2]), "=r"(r[O + 3]), "=r"(r[O + 4]), "=r"(r[O + 5]), "=r"(r[O + 6]),   \
        "=r"(r[O + 7]), "=r"(r[O + 8]), "=r"(r[O + 9]), "=r"(r[O + 10]), "=r"(r[O + 11]), "=r"(r[O + 12]),            \
        "=r"(r[O + 13]), "=r"(r[O + 14]), "=r"(r[O + 15])                                                             \
      : "r"(AT)                                                                                                       \
      : "memory")
    SGR_LD16(hi_at, 0);
    SGR_LD16(hi_at + apart, 16);
#undef SGR_LD16
    tmem_wait_ld32(r);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      hi[e] = __uint_as_float(r[e]);
      lo[e] = __uint_as_float(r[16 + e]);
    }
  }
}

// Whether a row sees a position (`last`, `row`: MassCtl's).
__device__ __forceinline__ bool mass_sees(const AttnParams& p, int pos, int first, int last, int row) {
  const int j = pos - first;
  if (p.tree && j >= 0) {
    if (last < 0 || (j >> 6) >= p.tree_words) return false;
    return (p.tree[row * p.tree_stride + (j >> 6)] >> (j & 63) & 1) != 0;
  }
  return row_sees(pos, last, p.window, p.sinks);
}

// Which of the rows from r on see a position (no tree): rows are in the order
// of their positions, so they are those from the position's own token on, up to
// the last whose window it is in.
__host__ __device__ __forceinline__ uint32_t mass_rows(const AttnParams& p, int pos, int first, int r, int rows) {
  const long long tok = (long long)pos - first;
  const long long lo = tok * p.group, hi = pos < p.sinks || p.window == INT_MAX ? rows : min((tok + p.window) * p.group, (long long)rows);
  const int a = (int)min(max(lo - r, 0LL), 32LL), b = (int)min(max(hi - r, 0LL), 32LL);  // columns [a, b)
  return a >= b ? 0u : (0xffffffffu >> (32 - b)) & (0xffffffffu << a);
}

template <int D, int NT>
__global__ void __launch_bounds__(MassShape<D, NT>::kThreads, 2)
    kv_mass_kernel(const __grid_constant__ CUtensorMap tmK, const MassParams mp) {
  using Sh = MassShape<D, NT>;
  constexpr int S = Sh::kStages, Q = Sh::kSlots, R = Sh::kRows, kCols = Sh::kCols, A = Sh::kAcc, kWeigh = Sh::kWeigh, kQuery = Sh::kQuery;
  const AttnParams& p = mp.a;
  extern __shared__ __align__(1024) unsigned char mass_smem[];
  const uint32_t base = smem_u32(mass_smem);
  if (base & 1023u) {  // swizzled operands could not be read
    pdl_wait();
    if (threadIdx.x == 0) report_error(p.err, kErrSmemAlign);
    return;
  }
  MassCtl<D, NT>& c = *reinterpret_cast<MassCtl<D, NT>*>(mass_smem);
  const uint32_t ring = base + mass_ctl_bytes<D, NT>(), qbuf = ring + S * Sh::kTileBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &c.abort;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&c.kfull[i]), 1);
      mbar_init(smem_u32(&c.empty[i]), 1 + kWeigh);  // the last product, the weighing warps
    }
    for (int i = 0; i < A; ++i) {
      mbar_init(smem_u32(&c.sfull[i]), 2);  // the product, and the thread that saw the page scales
      mbar_init(smem_u32(&c.sempty[i]), kWeigh);
    }
    for (int i = 0; i < Q; ++i) {
      mbar_init(smem_u32(&c.qfull[i]), kQuery);
      mbar_init(smem_u32(&c.qempty[i]), 1 + kWeigh);
    }
    mbar_init(smem_u32(&c.drain), 1);
    for (int i = 0; i < kAttnQueue; ++i) {
      mbar_init(smem_u32(&c.segfull[i]), 1);
      mbar_init(smem_u32(&c.segempty[i]), kWeigh + kQuery + 1);  // the weighing and query warps, the MMA thread
    }
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWeigh + 1) {
    tmem_alloc(smem_u32(&c.tmem), Sh::kTmemCols);
    tmem_relinquish();
  }
  if (tid == 32) prefetch_tmap(&tmK);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  // (only now: a dependent that allocates tensor memory must not come first)
  pdl_launch_dependents();
  pdl_wait();

  if (warp == kWeigh) {
    attn_walk<D, NT, true>(c, p, tmK, tmK, ring);
  } else if (warp == kWeigh + 1) {
    // ------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(kAttnTile, kCols);
      bool ok = true;
      auto need = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !mbar_wait_or_abort(smem_u32(bar), parity, abort_flag)) {
          if (!*abort_flag) report_error(p.err, kErrWaitFull);
          *abort_flag = 1;
          ok = false;
        }
        return ok;
      };
      int sq = 0, i = 0, x = 0, q0 = 0;  // segments, tiles, products, slots of queries before the segment's
      while (ok) {
        const int qi = sq % kAttnQueue;
        if (!need(&c.segfull[qi], (sq / kAttnQueue) & 1)) break;
        const int kind = c.seg[qi].kind, n = c.seg[qi].tb - c.seg[qi].ta, chunks = (c.seg[qi].nrows + R - 1) / R;
        mbar_arrive(smem_u32(&c.segempty[qi]));
        if (kind & kSegStop) break;
        ++sq;
        for (int t = 0; t < n && ok; ++t, ++i) {
          if (!need(&c.kfull[i % S], (i / S) & 1)) break;
          for (int k = 0; k < chunks; ++k, ++x) {
            const int q = (q0 + k) % Q;
            if (t == 0 && !need(&c.qfull[q], ((q0 + k) / Q) & 1)) break;
            if (!need(&c.sempty[x % A], ((x / A) & 1) ^ 1)) break;
            tc_fence_after();
            const uint64_t kd = smem_desc_rows<D>(ring + (uint32_t)(i % S) * Sh::kTileBytes);
            const uint64_t qd = smem_desc_rows<D>(qbuf + (uint32_t)q * Sh::kSlotBytes);
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              mma_e4m3(tmem + (uint32_t)(x % A) * kCols, kd + (uint64_t)(kk * 2), qd + (uint64_t)(kk * 2), idesc, kk > 0);
            mma_commit(smem_u32(&c.sfull[x % A]));
            mbar_arrive(smem_u32(&c.sfull[x % A]));
            if (k == chunks - 1) mma_commit(smem_u32(&c.empty[i % S]));
            if (t == n - 1) mma_commit(smem_u32(&c.qempty[q]));
          }
        }
        q0 += chunks;
      }
      mma_commit(smem_u32(&c.drain));
      if (!mbar_wait(smem_u32(&c.drain), 0)) report_error(p.err, kErrDrain);
    }
  } else if (warp >= kWeigh + 2) {
    // ----------------------------------------------------------- query operand
    constexpr int kLanes = D / 8, kStep = 32 * kQuery / kLanes, kPass = R / kStep;
    const int qt = tid - 32 * (kWeigh + 2), l = qt % kLanes;
    int sq = 0, slot = 0;
    uint32_t par = 0;
    bool ok = true;
    while (ok) {
      const int qi = sq % kAttnQueue;
      if (lane == 0) ok = mbar_wait_nap<kNap>(smem_u32(&c.segfull[qi]), (sq / kAttnQueue) & 1, abort_flag);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      const AttnSeg g = c.seg[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.segempty[qi]));
      ++sq;
      if (g.kind & kSegStop) break;
      for (int k = 0; k * R < g.nrows && ok; ++k) {
        // Row `pass` of this thread's: two are under way while one is converted.
        auto load_row = [&](int pass) {
          const int q = k * R + pass * kStep + qt / kLanes;
          if (q >= g.nrows) return make_uint4(0u, 0u, 0u, 0u);
          const int at = g.r0 + q, tok = div_group(p, at), head = g.h * p.group + at - tok * p.group;
          return *reinterpret_cast<const uint4*>(p.q.p + (long long)(g.row0 + tok) * p.q.ts + (long long)head * p.q.hs + 8 * l);
        };
        uint4 v0 = load_row(0), v1 = v0;
        if (kPass > 1) v1 = load_row(1);
        // What there is one of a row: a thread each.
        float lse = -INFINITY;
        int last = -1, row = 0;  // a row that is none sees nothing
        if (qt < R && k * R + qt < g.nrows) {
          const int at = g.r0 + k * R + qt, tok = div_group(p, at);
          row = g.row0 + tok;
          lse = p.lse[(long long)row * p.q.heads + g.h * p.group + at - tok * p.group];
          last = p.tree ? tree_row(p, g.row0, g.n, g.first, tok).last : row_last(g.first, tok);
        }
        if (lane == 0) ok = mbar_wait_nap<kNap>(smem_u32(&c.qempty[slot]), par ^ 1u, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
#pragma unroll 1
        for (int i = 0; i < kPass; ++i) {
          const int q = i * kStep + qt / kLanes;
          const uint4 v = v0;
          v0 = v1;
          if (i + 2 < kPass) v1 = load_row(i + 2);
          const QuerySplit s = split_query<kLanes>(v, 1.f, 32.f);
          const uint32_t qb = qbuf + (uint32_t)(slot * Sh::kSlotBytes) + (uint32_t)((l & 1) * 8);
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qb + swizzled<D>(q, l >> 1)), "r"(s.hi.x), "r"(s.hi.y) : "memory");
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qb + swizzled<D>(R + q, l >> 1)), "r"(s.lo.x), "r"(s.lo.y) : "memory");
          if (l == 0) c.qf[slot][q] = s.factor * p.scale_log2;
        }
        if (qt < R) {
          c.ql[slot][qt] = lse == -INFINITY ? -INFINITY : -1.4426950408889634f * lse;
          c.qpos[slot][qt] = last;
          c.qrow[slot][qt] = row;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.qfull[slot]));
        if (++slot == Q) {
          slot = 0;
          par ^= 1u;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- weights
    // After a wait that ran out (abort) the waits fall through, so that the
    // warps keep meeting at their barriers until the segments end.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar_wait_or_abort(smem_u32(bar), parity, abort_flag)) {
        if (!*abort_flag) report_error(p.err, kErrWaitMma);
        *abort_flag = 1;
      }
      __syncwarp();
    };
    // Group g of four warps takes columns C g .. C g + C - 1 of every product.
    constexpr int C = R / Sh::kGroups;
    const int group = warp >> 2, tok = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21) + (uint32_t)(group * C);  // tensor-memory lanes of this warp
    const int ps = p.cache.page_shift;
    int sq = 0, i = 0, x = 0, q0 = 0;
    while (true) {
      const int qi = sq % kAttnQueue;
      if (tid == 0) c.go[sq & 1] = mbar_wait_or_abort(smem_u32(&c.segfull[qi]), (sq / kAttnQueue) & 1, abort_flag) ? 1 : 0;
      __syncwarp();
      named_bar_sync(1, 32 * kWeigh);
      if (!c.go[sq & 1]) {
        if (tid == 0 && !*abort_flag) report_error(p.err, kErrWaitFull);
        *abort_flag = 1;
        break;
      }
      const AttnSeg g = c.seg[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.segempty[qi]));
      ++sq;
      if (g.kind & kSegStop) break;
      const TileMap tm(g.tlo, p.sinks);
      const int chunks = (g.nrows + R - 1) / R;
      if (g.n > mp.max_new && tid == 0) report_error(p.err, kErrIndex);
      const bool stray = !mp.part && g.r0 > 0;  // (rows that there is no room for)
      for (int t = g.ta; t < g.tb; ++t, ++i) {
        const int slot = i % S, pos = tm.at(t) * kAttnTile + tok;
        int flags = 0, page = -1;
        F2 key = f2(0.f, 0.f);
        bool live = false;
        F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        for (int k = 0; k < chunks; ++k, ++x) {
          const int q = (q0 + k) % Q, a = x % A;
          if (t == g.ta) wait(&c.qfull[q], ((q0 + k) / Q) & 1);
          wait(&c.sfull[a], (x / A) & 1);
          tc_fence_after();
          if (k == 0) {
            flags = c.flags[slot];
            page = c.page[slot][tok >> ps];
            key = f2(c.kscale[slot][tok >> ps], c.kscale[slot][tok >> ps]);
            live = page >= 0 && tok >= c.live[slot][0] && tok < c.live[slot][1];
          }
          const F2 third = f2(kLoScale, kLoScale);
          // Adds the weights of N columns from c0 on; seen: which count (kHide).
          auto weigh = [&](auto masked, const auto& hi, const auto& lo, int c0, uint32_t seen) {
            constexpr bool kHide = decltype(masked)::value;
            constexpr int N = sizeof(hi) / sizeof(float);
#pragma unroll
            for (int e = 0; e < N; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&c.qf[q][c0 + e]);
              const float4 l = *reinterpret_cast<const float4*>(&c.ql[q][c0 + e]);
              const F2 s0 = f2_fma(f2(lo[e], lo[e + 1]), third, f2(hi[e], hi[e + 1]));
              const F2 s1 = f2_fma(f2(lo[e + 2], lo[e + 3]), third, f2(hi[e + 2], hi[e + 3]));
              const float2 w0 = f2_parts(f2_fma(s0, f2_mul(f2(f.x, f.y), key), f2(l.x, l.y)));
              const float2 w1 = f2_parts(f2_fma(s1, f2_mul(f2(f.z, f.w), key), f2(l.z, l.w)));
              float w[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
              for (int m = 0; m < 4; ++m) w[m] = ex2(!kHide || (seen >> (e + m) & 1) ? w[m] : -INFINITY);
              sum[0] = f2_add(sum[0], f2(w[0], w[1]));
              sum[1] = f2_add(sum[1], f2(w[2], w[3]));
            }
          };
          const uint32_t cols = lanes + (uint32_t)(a * kCols);
          if (__builtin_expect(flags & 2, 0)) {  // (seldom: eight columns at a time, in as little code as that takes)
#pragma unroll 1
            for (int c0 = 0; c0 < C; c0 += 8) {
              float hi[8], lo[8];
              tmem_ld8x2(cols + (uint32_t)c0, cols + (uint32_t)(R + c0), hi, lo);
              const int at = group * C + c0;
              uint32_t seen = 0u;
              if (live && p.tree) {
#pragma unroll 1
                for (int e = 0; e < 8; ++e)
                  seen |= mass_sees(p, pos, g.first, c.qpos[q][at + e], c.qrow[q][at + e]) ? 1u << e : 0u;
              } else if (live) {
                seen = mass_rows(p, pos, g.first, g.r0 + k * R + at, g.r0 + g.nrows);
              }
              weigh(std::true_type(), hi, lo, at, seen);
            }
          } else {
            constexpr int P = C < 16 ? C : 16;  // columns at a time
#pragma unroll
            for (int c0 = 0; c0 < C; c0 += P) {
              float hi[P], lo[P];
              tmem_ld_parts<P>(cols + (uint32_t)c0, R, hi, lo);
              weigh(std::false_type(), hi, lo, group * C + c0, 0u);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&c.sempty[a]));
        }
        const float2 s2 = f2_parts(f2_add(sum[0], sum[1]));
        float w = s2.x + s2.y;
        if constexpr (Sh::kGroups > 1) {
          // Two buffers by the tile's parity: the second group, past the barrier of
          // tile i, may be at its sums of tile i + 1 while a warp of the first still
          // reads those of tile i; the barrier of tile i + 1, to which that warp comes
          // after its read, stands before the sums of tile i + 2.
          if (group > 0) c.sum[i & 1][tok] = w;
          __syncwarp();
          named_bar_sync(2, 32 * kWeigh);
          if (group == 0) w += c.sum[i & 1][tok];
        }
        if (!live) w = 0.f;
        if (group > 0 || stray) {
        } else if (mp.part) {
          mp.part[mass_part<NT>(mp, g.b, g.row0, g.r0 / NT, g.h) + pos] = w;
        } else if (live) {
          float* at = mp.mass + (long long)page * mp.page_stride + (long long)g.h * mp.head_stride + (pos & ((1 << ps) - 1));
          if (pos >= g.first)
            *at = w;
          else
            atomicAdd(at, w);  // (no read to wait for; the only one to this address but for pages that sequences share)
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.empty[slot]));
      }
      for (int k = 0; k < chunks; ++k)
        if (lane == 0) mbar_arrive(smem_u32(&c.qempty[(q0 + k) % Q]));
      q0 += chunks;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWeigh + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::kTmemCols);
  }
}

// Adds the row tiles' sums of a position, in order: block (x, y, z) takes tile x
// of sequence z and key/value head y, thread = position.
template <int NT>
__global__ void __launch_bounds__(kAttnTile) kv_mass_join_kernel(const MassParams mp) {
  const AttnParams& p = mp.a;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z, pos = (int)blockIdx.x * kAttnTile + (int)threadIdx.x;
  const KvSeq s = kv_seq(p.batch, p.cache.page_shift, b, nullptr);
  if (s.n == 0 || pos >= s.len) return;
  const long long at = mass_part<NT>(mp, b, s.row0, 0, h) + pos, step = (long long)p.cache.heads * mp.tiles * kAttnTile;
  float w = 0.f;
  bool any = false;
  // Eight sums are read at once, those that are not there from the last row tile's
  // place.  (Position by position: a tile that the rows see a part of may hold pages
  // that none of them sees, whose table entries may be anything.)
  constexpr int kRun = 8;
  const int count = (s.n * p.group + NT - 1) / NT;
  for (int j0 = 0; j0 < count; j0 += kRun) {
    float x[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) x[k] = mp.part[at + min(j0 + k, count - 1) * step];
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const AttnItem it = attn_item<NT, true>(p, s, j0 + k);
      if (j0 + k < count && pos < it.thi && (pos >= it.tlo || pos < p.sinks)) {
        w += x[k];
        any = true;
      }
    }
  }
  const int page = any ? p.batch.table[(long long)b * p.batch.table_stride + (pos >> p.cache.page_shift)] : -1;
  if (page < 0 || page >= p.cache.num_pages) return;  // (recorded by the kernel before)
  float* to = mp.mass + (long long)page * mp.page_stride + (long long)h * mp.head_stride + (pos & ((1 << p.cache.page_shift) - 1));
  if (pos >= s.len - s.n)
    *to = w;
  else
    atomicAdd(to, w);  // (other sequences may share the page; otherwise the only one to this address)
}

}  // namespace sgr
