// sgr_kv_evict.cuh -- eviction from the paged cache by accumulated attention
// weight (sgr_attention.h): which positions of a head stay, and their move to
// new pages.
//
// Bound: few positions: the chain of reads and cluster barriers (1100 positions:
// 10 us, of which the selection 6); one sequence of 130001: 40 us (selection 20,
// on 64 CTAs; the move 16, 67 MB); 48 of up to 8000 in pages of 16 by 64 codes, 417
// MB: 125 us (selection 25: additions to shared memory and issue; the move 78, 5.3
// TB/s under the profiler, issue slots 72% taken).
//
// Selection.  Of the positions between the protected ends the m with the
// largest mass stay, of equal ones the first.  Their masses as 32-bit keys in
// the order of the numbers, the m-th largest is found digit by digit (10, 11
// and 11 bits: a histogram of the keys that agree with the digits so far,
// summed from the top); the positions above it, and as many equal to it as are
// wanted, follow in one sweep in order.  A sequence's head is one cluster's
// work: each CTA has a run of positions, their keys in shared memory (read
// from global memory once; what does not fit is read again), and the
// histograms are added through distributed shared memory, so that one long
// sequence is not one CTA's.
//
// The move.  A block takes one new page of a head, K and V: positions' codes
// in registers, the largest magnitude over the page (each code under its old
// page's scale), the smallest power of two that holds it, and the codes to that
// scale: exact but for those that become subnormal.
#pragma once

#include <cstddef>
#include <type_traits>

#include "sgr_kv_attn.cuh"

namespace sgr {

struct EvictParams {
  KvCacheRef cache;
  KvBatch batch;  // (block table and lengths)
  float* mass;
  long long page_stride, head_stride;  // of the mass, elements
  const int* keep;
  const int* new_table;
  long long new_stride;
  int new_pages;
  int first, recent;
  int* kept;  // [batch][heads][new_pages << page_shift]
  int* new_len;
  int cached;  // keys that a CTA of the selection holds in shared memory
  int wide;    // whether 16-byte reads of the mass are aligned
  unsigned pages_inv, heads_inv;  // floor(2^32 / new_pages) and of the heads, at most 2^32 - 1
  unsigned* err;
};

constexpr int kSelectThreads = 512;
constexpr int kSelectCached = 32 * kSelectThreads;  // keys in shared memory at most
constexpr int kSelectCluster = 8;  // CTAs at most (the portable limit)

// Positions that stay: `first` at the beginning, `recent` at the end, `chosen`
// of the others.
struct EvictPlan {
  int len, first, recent, chosen;
  __device__ __forceinline__ int total() const { return first + chosen + recent; }
};

// n / d for 0 <= n < 2^31 by d's inverse: the product is at most one too small.
__device__ __forceinline__ int div_by(int n, int d, unsigned inv) {
  const int q = (int)__umulhi((unsigned)n, inv);
  return q + (n - q * d >= d ? 1 : 0);
}

__device__ __forceinline__ EvictPlan evict_plan(const EvictParams& p, int b, unsigned* err) {
  EvictPlan e;
  const long long room = (long long)p.batch.max_pages << p.cache.page_shift;
  const long long new_room = (long long)p.new_pages << p.cache.page_shift;
  const int len = p.batch.seq_len[b], keep = p.keep[b];
  e.len = len < 0 ? 0 : len > room ? (int)room : len;
  int n = min(max(keep, 0), e.len);
  const bool fits = n <= new_room;
  if (!fits) n = (int)new_room;
  if (e.len != len || keep < 0 || !fits) report_error(err, kErrIndex);
  e.first = min(p.first, n);
  e.recent = min(p.recent, n - e.first);
  e.chosen = n - e.first - e.recent;
  return e;
}

// The order of numbers as that of unsigned ones: -0 as 0, NaN above all.  No
// number has the keys 0 and 1.
constexpr uint32_t kKeyNone = 0, kKeyBadPage = 1;

__device__ __forceinline__ uint32_t mass_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

struct alignas(16) SelectCtl {
  static constexpr int kWarps = kSelectThreads / 32;
  // Histograms of the digits over the cluster, each CTA the sums of its share of
  // the bins.  Masses crowd in a few bins of the first digit: each CTA counts its
  // own there before, in four copies by lane.
  unsigned own[1 << 10][4], sum0[1 << 10], sum1[1 << 11], sum2[1 << 11];
  unsigned pick[2], warp_sum[kWarps];
  int counts[2];  // of this CTA: above the threshold, at it
  int warp_above[kWarps], warp_equal[kWarps];
  // (the keys follow)
};

// A CTA's run of a sequence, from position lo on: those of i0 <= i < i1 are to be
// chosen from.
struct SelectRun {
  const int* table;
  const float* of_head;  // masses of page 0
  long long lo;
  int i0, i1;
};

// The keys of N groups of four positions, `step` apart; kKeyNone for those that
// are not to be chosen from.  Two round trips, the table's and the masses'
// (pages have multiples of 16 positions).
template <int N>
__device__ __forceinline__ void select_load(const EvictParams& p, const SelectRun& r, int at0, int step, uint4 (&out)[N]) {
  const int ps = p.cache.page_shift;
  int page[N];
  float v[N][4];
  const int last = (r.i1 - 1) & ~3, begin = r.i0 & ~3;  // (a group beyond the run reads its last one)
#pragma unroll
  for (int k = 0; k < N; ++k) page[k] = r.table[(int)(r.lo + max(min(at0 + k * step, last), begin)) >> ps];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int pos = (int)(r.lo + max(min(at0 + k * step, last), begin));
    const bool there = page[k] >= 0 && page[k] < p.cache.num_pages;
    const float* at = r.of_head + (there ? page[k] : 0) * p.page_stride + (pos & ((1 << ps) - 1));
    if (p.wide) {
      const float4 x = *reinterpret_cast<const float4*>(at);
      v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) v[k][m] = at[m];
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = at0 + k * step;
    const bool there = page[k] >= 0 && page[k] < p.cache.num_pages;
    if (!there && i < r.i1 && i + 4 > r.i0) report_error(p.err, kErrIndex);
    uint32_t u[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
      u[m] = i + m < r.i0 || i + m >= r.i1 ? kKeyNone : there ? mass_key(v[k][m]) : kKeyBadPage;
    out[k] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const EvictParams p) {
  constexpr int kWarps = SelectCtl::kWarps;
  extern __shared__ __align__(16) unsigned char select_smem[];
  SelectCtl& s = *reinterpret_cast<SelectCtl*>(select_smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(select_smem + sizeof(SelectCtl));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned ranks, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
  rank = cluster_ctarank();
  for (int i = tid; i < (int)(offsetof(SelectCtl, pick) / 16); i += kSelectThreads)
    reinterpret_cast<uint4*>(select_smem)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (ranks > 1) cluster_arrive();  // (the sums are zeros: others may add to them behind the wait)
  pdl_launch_dependents();
  pdl_wait();
  const int item = (int)(blockIdx.x / ranks), h = item % p.cache.heads, b = item / p.cache.heads;
  const EvictPlan e = evict_plan(p, b, p.err);
  const int ps = p.cache.page_shift, span = e.len - e.first - e.recent;  // positions to choose from
  // This CTA's run of the sequence, whole groups of four positions: those with
  // lo <= i0, i1 (relative to it) are to be chosen from.
  const int chunk = (int)((((long long)e.len + ranks - 1) / ranks + 3) & ~3LL);
  const long long lo = (long long)chunk * rank;
  const int i0 = (int)min(max(e.first - lo, 0LL), (long long)chunk);
  const int i1 = max((int)min((long long)(e.len - e.recent) - lo, (long long)chunk), i0);
  const int* table = p.batch.table + (long long)b * p.batch.table_stride;
  const float* of_head = p.mass + (long long)h * p.head_stride;
  int* kept = p.kept + (long long)item * ((long long)p.new_pages << ps);
  // The protected ends.
  for (int i = (int)rank * kSelectThreads + tid; i < e.first + e.recent; i += (int)ranks * kSelectThreads) {
    if (i < e.first)
      kept[i] = i;
    else
      kept[i + e.chosen] = e.len - e.recent + (i - e.first);
  }
  if (h == 0 && rank == 0 && tid == 0) p.new_len[b] = e.total();
  const bool all = e.chosen == span;
  if (all) {
    for (int i = i0 + tid; i < i1; i += kSelectThreads) kept[lo + i] = (int)lo + i;
  }
  if (all || e.chosen == 0) {  // (every CTA of the cluster)
    if (ranks > 1) cluster_wait();
    return;
  }
  const SelectRun r{table, of_head, lo, i0, i1};
  // (a CTA without positions to choose from takes part in the sums with none)
  const int end = i1 > i0 ? (i1 + 3) & ~3 : 0, cached = min(end, p.cached);
  for (int i = 4 * tid; i < cached; i += 8 * 4 * kSelectThreads) {
    uint4 u[8];
    select_load(p, r, i, 4 * kSelectThreads, u);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k * 4 * kSelectThreads < cached) *reinterpret_cast<uint4*>(keys + i + k * 4 * kSelectThreads) = u[k];
  }
  auto key4 = [&](int i) {
    if (i < p.cached) return *reinterpret_cast<const uint4*>(keys + i);
    uint4 u[1];
    select_load(p, r, i, 0, u);
    return u[0];
  };
  // Every thread's keys, in fours.
  auto each = [&](auto f) {
#pragma unroll 2
    for (int i = 4 * tid; i < end; i += 4 * kSelectThreads) {
      const uint4 u = key4(i);
      f(u.x), f(u.y), f(u.z), f(u.w);
    }
  };
  __syncthreads();
  // ------------------------------------------------------------ the threshold
  uint32_t prefix = 0;                 // the digits found so far
  unsigned want = (unsigned)e.chosen;  // of the keys that agree with them, the largest
  // Adds to a bin's sum in the CTA that has it.
  const int share = __ffs(ranks) - 1;  // (a power of two)
  auto add = [&](unsigned* sum, int log_bins, uint32_t bin, unsigned count) {
    if (ranks == 1)
      atomicAdd(sum + bin, count);
    else
      asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(
                       map_to_rank(smem_u32(sum + bin), bin >> (log_bins - share))),
                   "r"(count)
                   : "memory");
  };
  auto meet = [&] {
    if (ranks > 1)
      cluster_sync_all();
    else
      __syncthreads();
  };
  // Finds the bin in which, from the highest down, the wanted number is reached.
  auto find = [&](auto log_bins_of, const unsigned* sum) {
    constexpr int kLog = decltype(log_bins_of)::value, kMine = (1 << kLog) / kSelectThreads;
    static_assert(kMine == 2 || kMine == 4, "a thread reads its bins at once, on their own alignment");
    meet();  // (every CTA's counts)
    const int top = (1 << kLog) - kMine * (tid + 1);  // this thread's bins, from the highest ones down
    unsigned c[4] = {0u, 0u, 0u, 0u};
    const uint32_t at = map_to_rank(smem_u32(sum + top), (uint32_t)top >> (kLog - share));
    if constexpr (kMine == 4)
      asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]) : "r"(at) : "memory");
    else
      asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(c[0]), "=r"(c[1]) : "r"(at) : "memory");
    const unsigned mine = c[0] + c[1] + c[2] + c[3];
    unsigned upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    if (lane == 31) s.warp_sum[warp] = upto;
    __syncthreads();
    unsigned above = upto - mine + __reduce_add_sync(0xffffffffu, lane < warp ? s.warp_sum[lane % kWarps] : 0u);
#pragma unroll
    for (int k = kMine - 1; k >= 0; --k) {
      if (above < want && want <= above + c[k]) {
        s.pick[0] = (unsigned)(top + k);
        s.pick[1] = want - above;
      }
      above += c[k];
    }
    __syncthreads();
    want = s.pick[1];
    return s.pick[0];
  };
  each([&](uint32_t u) {
    if (u != kKeyNone) atomicAdd(&s.own[u >> 22][lane & 3], 1u);
  });
  if (ranks > 1) cluster_wait();
  __syncthreads();
  for (int i = tid; i < 1 << 10; i += kSelectThreads) {
    const uint4 c = *reinterpret_cast<const uint4*>(s.own[i]);
    const unsigned n = c.x + c.y + c.z + c.w;
    if (n) add(s.sum0, 10, i, n);
  }
  prefix = find(std::integral_constant<int, 10>(), s.sum0);
  // (kKeyNone is below every key and the sums begin at the top: counted or not,
  // it is never reached)
  each([&](uint32_t u) {
    if (u >> 22 == prefix) add(s.sum1, 11, u >> 11 & 0x7FF, 1u);
  });
  prefix = prefix << 11 | find(std::integral_constant<int, 11>(), s.sum1);
  each([&](uint32_t u) {
    if (u >> 11 == prefix) add(s.sum2, 11, u & 0x7FF, 1u);
  });
  prefix = prefix << 11 | find(std::integral_constant<int, 11>(), s.sum2);
  // --------------------------------------------------------------- the positions
  // Each warp takes a run of the CTA's, a lane four neighbours at a time; `want`
  // of the keys equal to the threshold, the first, are taken.
  const int run = ((end + kWarps - 1) / kWarps + 127) / 128 * 128, w0 = min(warp * run, end), w1 = min(w0 + run, end);
  int above = 0, equal = 0;
  for (int i = w0 + 4 * lane; i < w1; i += 128) {
    const uint4 u = key4(i);
    above += (u.x > prefix) + (u.y > prefix) + (u.z > prefix) + (u.w > prefix);
    equal += (u.x == prefix) + (u.y == prefix) + (u.z == prefix) + (u.w == prefix);
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    s.warp_above[warp] = above;
    s.warp_equal[warp] = equal;
  }
  __syncthreads();
  if (tid == 0) {
    int a = 0, q = 0;
    for (int w = 0; w < kWarps; ++w) a += s.warp_above[w], q += s.warp_equal[w];
    s.counts[0] = a;
    s.counts[1] = q;
  }
  meet();
  int before_above = 0, before_equal = 0;  // in the CTAs, then in the warps before
  for (unsigned r = 0; r < rank; ++r) {
    const uint32_t at = map_to_rank(smem_u32(s.counts), r);
    int x, y;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(at) : "memory");
    before_above += x;
    before_equal += y;
  }
  if (ranks > 1) cluster_arrive();
  for (int w = 0; w < warp; ++w) before_above += s.warp_above[w], before_equal += s.warp_equal[w];
  for (int i = w0 + 4 * lane; i - 4 * lane < w1; i += 128) {
    uint4 x = make_uint4(kKeyNone, kKeyNone, kKeyNone, kKeyNone);
    if (i < w1) x = key4(i);
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    int mine = 0;  // above, and equal in the upper half
#pragma unroll
    for (int m = 0; m < 4; ++m) mine += (u[m] > prefix ? 1 : 0) + (u[m] == prefix ? 1 << 16 : 0);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    const int all_of = __shfl_sync(0xffffffffu, upto, 31);
    int ov = before_above + ((upto - mine) & 0xFFFF), eq = before_equal + ((upto - mine) >> 16);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (u[m] > prefix || (u[m] == prefix && eq < (int)want)) kept[e.first + ov + min(eq, (int)want)] = (int)lo + i + m;
      ov += u[m] > prefix ? 1 : 0;
      eq += u[m] == prefix ? 1 : 0;
    }
    before_above += all_of & 0xFFFF;
    before_equal += all_of >> 16;
  }
  if (ranks > 1) cluster_wait();  // (until all have read this CTA's counts)
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Largest magnitude of 16 codes, as its code (NaN does not count).
__device__ __forceinline__ uint32_t largest_code(const uint4& v) {
  uint32_t u[4] = {v.x & 0x7F7F7F7Fu, v.y & 0x7F7F7F7Fu, v.z & 0x7F7F7F7Fu, v.w & 0x7F7F7F7Fu};
  const uint32_t nan = (u[0] + 0x01010101u) | (u[1] + 0x01010101u) | (u[2] + 0x01010101u) | (u[3] + 0x01010101u);
  if (__builtin_expect(nan & 0x80808080u, 0)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] &= ~__vcmpeq4(u[j], 0x7F7F7F7Fu);
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max_u16x2(max_u16x2(m, u[j] & 0x00FF00FFu), u[j] >> 8 & 0x00FF00FFu);
  return max(m & 0xFFFFu, m >> 16);
}

// 2^d as a pair of FP16 numbers, -24 <= d <= 15.
__device__ __forceinline__ uint32_t f16x2_exp2(int d) {
  const uint32_t h = d >= -14 ? (uint32_t)(d + 15) << 10 : 1u << (24 + d);
  return h | h << 16;
}

// Four codes times 2^d as f = f16x2_exp2(d), rounded to codes.  In FP16 a code
// times a power of two is exact down to multiples of 2^-24, far below what E4M3
// rounds to zero, and the factor 2^-24 rounds all codes to zero, as lesser ones do.
__device__ __forceinline__ uint32_t scale_codes(uint32_t v, uint32_t f) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 x, y;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 x, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, hi;\n\t"
      "mul.rn.f16x2 x, x, %2;\n\t"
      "mul.rn.f16x2 y, y, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 lo, x;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 hi, y;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "r"(v), "r"(f));
  return r;
}

constexpr int kMoveThreads = 256;

// A warp holds kVec 16-byte runs a lane of K and of V: kTok positions, whose
// numbers, pages, scales and masses are one lane's each.  A page's head is the
// work of as many warps as that takes (one for 16 positions of 64 codes, eight
// for 128 of 128), so that all lanes have reads under way.
template <int D, int kVec>
__global__ void __launch_bounds__(kMoveThreads, kVec == 2 ? 6 : 4) kv_move_kernel(const EvictParams p) {
  constexpr int kLanes = D / 16, kTok = 32 * kVec / kLanes;  // lanes of a position
  __shared__ float part[2][kMoveThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int ps = p.cache.page_shift, heads = p.cache.heads;
  const int warps = max((1 << ps) / kTok, 1), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shift = __ffs(warps) - 1;  // (a power of two)
  const int units = p.batch.batch * heads * p.new_pages, all = (int)blockIdx.x * (kMoveThreads / 32 >> shift) + (warp >> shift);
  const int unit = min(all, units - 1), item = div_by(unit, p.new_pages, p.pages_inv), block = unit - item * p.new_pages;
  const int b = div_by(item, heads, p.heads_inv), h = item - b * heads, slot0 = block << ps, t0 = (warp & (warps - 1)) * kTok;
  // (three round trips: the number of positions, which, and the new page; their
  // pages; what they hold.  Positions past the number may be read, not followed.)
  int count = all < units ? min(p.new_len[b] - slot0, 1 << ps) : 0;
  const int to = p.new_table[(long long)b * p.new_stride + block];
  const int mine = t0 + min(lane, kTok - 1);  // this lane's position of the new page
  int from = p.kept[(long long)item * ((long long)p.new_pages << ps) + slot0 + mine];
  if (count > 0 && (to < 0 || to >= p.cache.num_pages)) {
    if (lane == 0) report_error(p.err, kErrIndex);
    count = 0;
  }
  int page = -1;
  if (mine < count) {
    page = p.batch.table[(long long)b * p.batch.table_stride + (from >> ps)];
    if (page < 0 || page >= p.cache.num_pages) {
      report_error(p.err, kErrIndex);
      page = -1;
    }
  }
  from &= (1 << ps) - 1;
  uint4 v[2][kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int tok = (i * 32 + lane) / kLanes;
    const int of = __shfl_sync(0xffffffffu, page, tok), off = __shfl_sync(0xffffffffu, from, tok);
    v[0][i] = v[1][i] = make_uint4(0u, 0u, 0u, 0u);
    if (of < 0) continue;
    const long long at = of * p.cache.page_stride + h * p.cache.head_stride + off * p.cache.token_stride + lane % kLanes * 16;
    v[0][i] = *reinterpret_cast<const uint4*>(p.cache.k + at);
    v[1][i] = *reinterpret_cast<const uint4*>(p.cache.v + at);
  }
  float scale[2] = {1.f, 1.f}, mass = 0.f;
  if (page >= 0) {
    scale[0] = p.cache.k_scale[page * p.cache.scale_stride + h];
    scale[1] = p.cache.v_scale[page * p.cache.scale_stride + h];
    mass = p.mass[page * p.page_stride + h * p.head_stride + from];
  }
  int e_old[2], e_new[2];
  float top[2] = {0.f, 0.f};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    e_old[x] = min(max((int)(__float_as_uint(scale[x]) >> 23 & 0xFF) - 127, kKvExpMin), kKvExpMax);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      float a0, a1, a2, a3;
      from_e4m3x4(largest_code(v[x][i]), a0, a1, a2, a3);
      top[x] = fmaxf(top[x], a0 * kv_exp2i(__shfl_sync(0xffffffffu, e_old[x], (i * 32 + lane) / kLanes)));
    }
    top[x] = warp_max(top[x]);
    if (lane == 0) part[x][warp] = top[x];
  }
  if (warps > 1) {
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x)
      for (int w = warp & ~(warps - 1); w < (warp & ~(warps - 1)) + warps; ++w) top[x] = fmaxf(top[x], part[x][w]);
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) e_new[x] = kv_scale_exp(top[x]);
  const long long page_at = to * p.cache.page_stride + h * p.cache.head_stride;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int tok = (i * 32 + lane) / kLanes, t = t0 + tok;
    const long long at = page_at + t * p.cache.token_stride + lane % kLanes * 16;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int e = __shfl_sync(0xffffffffu, e_old[x], tok);
      uint32_t u[4] = {v[x][i].x, v[x][i].y, v[x][i].z, v[x][i].w};
      if (e != e_new[x]) {
        const int d = e - e_new[x];
        const uint32_t f = f16x2_exp2(max(min(d, 15), -24));
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = scale_codes(u[j], f);
        if (__builtin_expect(d > 15, 0)) {  // (2^17 at most for codes other than zero)
#pragma unroll
          for (int j = 0; j < 4; ++j) u[j] = scale_codes(u[j], f16x2_exp2(min(d - 15, 15)));
        }
      }
      if (t < count) *reinterpret_cast<uint4*>((x ? p.cache.v : p.cache.k) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
  if (lane < kTok && mine < count) p.mass[to * p.page_stride + h * p.head_stride + mine] = mass;
  if (count > 0 && t0 == 0 && lane < 2)
    (lane ? p.cache.v_scale : p.cache.k_scale)[to * p.cache.scale_stride + h] = kv_exp2i(lane ? e_new[1] : e_new[0]);
}

}  // namespace sgr
