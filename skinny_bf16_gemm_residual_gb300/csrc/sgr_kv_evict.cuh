// sgr_kv_evict.cuh -- eviction from the paged cache by accumulated attention
// weight (sgr_attention.h): which positions of a head stay, and their move to
// new pages.
//
// Selection.  Of the positions between the protected ends the m with the
// largest mass stay, of equal ones the first.  Their masses as 32-bit keys in
// the order of the numbers, the m-th largest is found digit by digit (11, 11
// and 10 bits: a histogram of the keys that agree with the digits so far,
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

#include "sgr_kv_append.cuh"

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
  unsigned* err;
};

constexpr int kSelectThreads = 512, kSelectCached = 16384, kSelectBins = 2048;
constexpr int kSelectCluster = 8;  // CTAs at most (the portable limit)

// Positions that stay: `first` at the beginning, `recent` at the end, `chosen`
// of the others.
struct EvictPlan {
  int len, first, recent, chosen;
  __device__ __forceinline__ int total() const { return first + chosen + recent; }
};

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

// The order of numbers as that of unsigned ones: -0 as 0, NaN above all.
__device__ __forceinline__ uint32_t mass_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

struct SelectCtl {
  static constexpr int kWarps = kSelectThreads / 32;
  unsigned hist[3][kSelectBins];  // of each digit
  uint32_t keys[kSelectCached];
  unsigned pick[2], warp_sum[kWarps];
  int counts[2];  // of this CTA: above the threshold, at it
  int warp_above[kWarps], warp_equal[kWarps];
};

__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const EvictParams p) {
  constexpr int kWarps = SelectCtl::kWarps;
  extern __shared__ __align__(16) unsigned char select_smem[];
  SelectCtl& s = *reinterpret_cast<SelectCtl*>(select_smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned ranks, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
  rank = cluster_ctarank();
  for (int i = tid; i < 3 * kSelectBins; i += kSelectThreads) (&s.hist[0][0])[i] = 0u;
  pdl_launch_dependents();
  pdl_wait();
  const int item = (int)(blockIdx.x / ranks), h = item % p.cache.heads, b = item / p.cache.heads;
  const EvictPlan e = evict_plan(p, b, p.err);
  const int ps = p.cache.page_shift, span = e.len - e.first - e.recent;  // positions to choose from
  // This CTA's run of them, whole warps of positions to each warp.
  const int chunk = (int)(((long long)span + ranks - 1) / ranks), lo = e.first + min((long long)chunk * rank, (long long)span);
  const int n = min(chunk, e.first + span - lo);
  const int* table = p.batch.table + (long long)b * p.batch.table_stride;
  auto load = [&](int i) {
    const int pos = lo + i, page = table[pos >> ps];
    if (page < 0 || page >= p.cache.num_pages) {
      report_error(p.err, kErrIndex);
      return 0u;
    }
    return mass_key(p.mass[(long long)page * p.page_stride + (long long)h * p.head_stride + (pos & ((1 << ps) - 1))]);
  };
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
    for (int i = tid; i < n; i += kSelectThreads) kept[lo + i] = lo + i;
    return;  // (every CTA of the cluster)
  }
  if (e.chosen == 0) return;
  const int cached = min(n, kSelectCached);
#pragma unroll 4
  for (int i = tid; i < cached; i += kSelectThreads) s.keys[i] = load(i);
  auto key = [&](int i) { return i < kSelectCached ? s.keys[i] : load(i); };
  __syncthreads();
  // ------------------------------------------------------------ the threshold
  uint32_t prefix = 0;               // the digits found so far
  unsigned want = (unsigned)e.chosen;  // of the keys that agree with them, the largest
  constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll
  for (int d = 0; d < 3; ++d) {
    const uint32_t mask = (1u << kBits[d]) - 1u;
    for (int i = tid; i < n; i += kSelectThreads) {
      const uint32_t u = key(i);
      if (d == 0 || u >> (kShift[d] + kBits[d]) == prefix) atomicAdd(&s.hist[d][u >> kShift[d] & mask], 1u);
    }
    cluster_sync_all();  // (every CTA's counts)
    // Four bins a thread, the highest first: bins 2047 - 4 tid and below.
    const int top = kSelectBins - 4 - 4 * tid;
    unsigned c[4] = {0u, 0u, 0u, 0u};
    for (unsigned r = 0; r < ranks; ++r) {
      const uint32_t at = map_to_rank(smem_u32(&s.hist[d][top]), r);
      unsigned v[4];
      asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                   : "r"(at)
                   : "memory");
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] += v[k];
    }
    const unsigned mine = c[0] + c[1] + c[2] + c[3];
    unsigned upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    if (lane == 31) s.warp_sum[warp] = upto;
    __syncthreads();
    unsigned above = upto - mine;
    for (int w = 0; w < warp; ++w) above += s.warp_sum[w];
#pragma unroll
    for (int k = 3; k >= 0; --k) {  // the bin in which the wanted number is reached
      if (above < want && want <= above + c[k]) {
        s.pick[0] = (unsigned)(top + k);
        s.pick[1] = want - above;
      }
      above += c[k];
    }
    __syncthreads();
    prefix = prefix << kBits[d] | s.pick[0];
    want = s.pick[1];
    __syncthreads();
  }
  // --------------------------------------------------------------- the positions
  // Each warp takes a run of the CTA's; `want` of the keys equal to the
  // threshold, the first, are taken.
  const int run = ((n + kWarps - 1) / kWarps + 31) / 32 * 32, i0 = min(warp * run, n), i1 = min(i0 + run, n);
  int above = 0, equal = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t u = key(i);
    above += u > prefix ? 1 : 0;
    equal += u == prefix ? 1 : 0;
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
  cluster_sync_all();
  int before_above = 0, before_equal = 0;  // in the CTAs, then in the warps before
  for (unsigned r = 0; r < rank; ++r) {
    const uint32_t at = map_to_rank(smem_u32(s.counts), r);
    int x, y;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(at) : "memory");
    before_above += x;
    before_equal += y;
  }
  cluster_arrive();
  for (int w = 0; w < warp; ++w) before_above += s.warp_above[w], before_equal += s.warp_equal[w];
  for (int i = i0; i < i1; i += 32) {
    const bool there = i + lane < i1;
    const uint32_t u = there ? key(i + lane) : 0u;
    const bool over = there && u > prefix, same = there && u == prefix;
    const unsigned eq = __ballot_sync(0xffffffffu, same), lower = (1u << lane) - 1u;
    const bool take = over || (same && before_equal + __popc(eq & lower) < (int)want);
    const unsigned ov = __ballot_sync(0xffffffffu, over);
    if (take) {
      const int at = before_above + __popc(ov & lower) + min(before_equal + __popc(eq & lower), (int)want);
      kept[e.first + at] = lo + i + lane;
    }
    before_above += __popc(ov);
    before_equal += __popc(eq);
  }
  cluster_wait();  // (until all have read this CTA's counts)
}

// Largest magnitude of 16 codes, as its code (NaN does not count).
__device__ __forceinline__ uint32_t largest_code(const uint4& v) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = u[j] & 0x7F7F7F7Fu;
    m = __vmaxu4(m, a & ~__vcmpeq4(a, 0x7F7F7F7Fu));
  }
  m = __vmaxu4(m, m >> 16);
  return max(m & 0xFFu, m >> 8 & 0xFFu);
}

constexpr int kMoveThreads = 256;

// kPass: positions of a page that a thread holds (16 codes of each).
template <int D, int kPass>
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const EvictParams p) {
  constexpr int kLanes = D / 16, kTok = kMoveThreads / kLanes;
  __shared__ float part[2][kMoveThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int ps = p.cache.page_shift, heads = p.cache.heads;
  const int block = (int)(blockIdx.x % (unsigned)p.new_pages), item = (int)(blockIdx.x / (unsigned)p.new_pages);
  const int h = item % heads, b = item / heads, slot0 = block << ps;
  const int count = min(p.new_len[b] - slot0, 1 << ps);
  if (count <= 0) return;
  const int to = p.new_table[(long long)b * p.new_stride + block];
  if (to < 0 || to >= p.cache.num_pages) {
    if (threadIdx.x == 0) report_error(p.err, kErrIndex);
    return;
  }
  const int* kept = p.kept + (long long)item * ((long long)p.new_pages << ps) + slot0;
  const int* table = p.batch.table + (long long)b * p.batch.table_stride;
  const int l = threadIdx.x % kLanes, tok = threadIdx.x / kLanes, lane = threadIdx.x & 31;
  uint4 v[2][kPass];
  int e_old[2][kPass];
  float gathered[kPass];
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int t = i * kTok + tok;
    v[0][i] = v[1][i] = make_uint4(0u, 0u, 0u, 0u);
    e_old[0][i] = e_old[1][i] = 0;
    gathered[i] = 0.f;
    if (t >= count) continue;
    const int pos = kept[t], page = table[pos >> ps], off = pos & ((1 << ps) - 1);
    if (page < 0 || page >= p.cache.num_pages) {
      report_error(p.err, kErrIndex);
      continue;
    }
    const long long at = (long long)page * p.cache.page_stride + (long long)h * p.cache.head_stride +
                         (long long)off * p.cache.token_stride + l * 16;
    v[0][i] = *reinterpret_cast<const uint4*>(p.cache.k + at);
    v[1][i] = *reinterpret_cast<const uint4*>(p.cache.v + at);
    const long long sc = (long long)page * p.cache.scale_stride + h;
    e_old[0][i] = (int)(__float_as_uint(p.cache.k_scale[sc]) >> 23 & 0xFF) - 127;
    e_old[1][i] = (int)(__float_as_uint(p.cache.v_scale[sc]) >> 23 & 0xFF) - 127;
    if (l == 0) gathered[i] = p.mass[(long long)page * p.page_stride + (long long)h * p.head_stride + off];
  }
  int e_new[2];
  float top[2] = {0.f, 0.f};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      float a0, a1, a2, a3;
      from_e4m3x4(largest_code(v[x][i]), a0, a1, a2, a3);
      e_old[x][i] = min(max(e_old[x][i], kKvExpMin), kKvExpMax);
      top[x] = fmaxf(top[x], a0 * kv_exp2i(e_old[x][i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], o));
    if (lane == 0) part[x][threadIdx.x >> 5] = top[x];
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
#pragma unroll
    for (int w = 0; w < kMoveThreads / 32; ++w) top[x] = fmaxf(top[x], part[x][w]);
    e_new[x] = kv_scale_exp(top[x]);
  }
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int t = i * kTok + tok;
    if (t >= count) break;
    const long long at = (long long)to * p.cache.page_stride + (long long)h * p.cache.head_stride +
                         (long long)t * p.cache.token_stride + l * 16;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t u[4] = {v[x][i].x, v[x][i].y, v[x][i].z, v[x][i].w};
      if (e_old[x][i] != e_new[x]) {
        // (a page of zeros has the least scale: zeros times 2^127 stay zeros)
        const float f = kv_exp2i(min(e_old[x][i] - e_new[x], 127));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float a0, a1, a2, a3;
          from_e4m3x4(u[j], a0, a1, a2, a3);
          u[j] = to_e4m3x4(a0 * f, a1 * f, a2 * f, a3 * f);
        }
      }
      *reinterpret_cast<uint4*>((x ? p.cache.v : p.cache.k) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    }
    if (l == 0) p.mass[(long long)to * p.page_stride + (long long)h * p.head_stride + t] = gathered[i];
  }
  if (threadIdx.x < 2)
    (threadIdx.x ? p.cache.v_scale : p.cache.k_scale)[(long long)to * p.cache.scale_stride + h] = kv_exp2i(e_new[threadIdx.x]);
}

}  // namespace sgr
