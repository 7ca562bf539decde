// sgr_kv_append.cuh -- norm and rotation of query and key heads, and the
// append of keys and values to the paged E4M3 cache (sgr_attention.h).
//
// A head is D / 8 lanes of 8 elements: the norm is one sum of squares in FP32
// over them, 1 / sqrt(mean + eps) and the weight multiply it, and each lane
// holds both elements of its four pairs, so that the rotation needs no
// exchange.  One rounding, to BF16 or E4M3, at the end.
//
// A scale is a power of two: x / s is then exact, and a page whose scale grows
// has its earlier codes divided by a power of two, exact but for those that
// become subnormal.  The price is up to one of E4M3's 15 binades of range.
//
// One launch does all of an append: the first blocks take query rows, the
// others one (page, key/value head, K or V) each.  A block that owns a page's
// head needs no atomics for its scale: it holds the page's new tokens in
// registers, finds their largest magnitude, and then writes codes and scale.
//
// Bound: for prompts neither memory (each input read once, each output written
// once) nor issue slots are full, both are used for most of the time; for a
// handful of rows the chain of dependent loads.  Measured: norm + rotation of
// 12345 rows of 72 heads (458 MB) 88-90 us, 5.1 TB/s, issue slots 67% taken; of
// 16 rows of 32 heads 1.4 us.  Append of 6012 prompt rows of 64 + 8 + 8 heads
// (237 MB) 51 us, 4.6 TB/s, issue slots 73% taken; of one row 2.7 us, of 48
// rows 4.9.  More blocks an SM (fewer registers) or packed FP32 arithmetic
// (more registers) were slower for the append, and within 4% for the norm.
#pragma once

#include "sgr_kv_common.cuh"

namespace sgr {

// Exponent of the smallest power of two s with amax <= 448 s (448 = 1.75 2^8).
__device__ __forceinline__ int kv_scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kKvExpMin), kKvExpMax);  // amax = 0 and subnormals: the least scale
}

__device__ __forceinline__ float kv_exp2i(int e) { return __int_as_float((max(e, -126) + 127) << 23); }

__device__ __forceinline__ uint32_t to_e4m3x4(float a0, float a1, float a2, float a3) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a0), "f"(a1), "f"(a2), "f"(a3));
  return r;
}

__device__ __forceinline__ void from_e4m3x4(uint32_t v, float& a0, float& a1, float& a2, float& a3) {
  asm("{\n\t.reg .b16 lo, hi, x0, x1, x2, x3;\n\t.reg .b32 h01, h23;\n\t"
      "mov.b32 {lo, hi}, %4;\n\t"
      "cvt.rn.f16x2.e4m3x2 h01, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 h23, hi;\n\t"
      "mov.b32 {x0, x1}, h01;\n\t"
      "mov.b32 {x2, x3}, h23;\n\t"
      "cvt.f32.f16 %0, x0;\n\tcvt.f32.f16 %1, x1;\n\tcvt.f32.f16 %2, x2;\n\tcvt.f32.f16 %3, x3;\n\t}"
      : "=f"(a0), "=f"(a1), "=f"(a2), "=f"(a3)
      : "r"(v));
}

// ------------------------------------------------------------- norm + rotation
constexpr int kRopeThreads = 128;

struct RopeParams {
  KvHeads q, k, qo, ko;
  const int* positions;
  NormRope nr;
  unsigned* err;
  int heads_per_block, q_chunks;  // of a block, and blocks of a row's query heads
};

// kPass passes of the block's warps over heads h0, h0 + 1, ... of one row of
// src, D / 8 lanes a head.  All passes' reads are asked for first; the lanes
// keep their pairs' cosines and sines and their weights over the heads.
template <int D, int kPass>
__device__ __forceinline__ void rope_row(const KvHeads& src, const KvHeads& dst, const __nv_bfloat16* weight,
                                         const NormRope& nr, int row, int pos, int h0, unsigned* err) {
  constexpr int kPerWarp = 32 / (D / 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, step = (int)(blockDim.x >> 5) * kPerWarp;
  const HeadLane<D> hl(lane, nr.rot, nr.interleaved != 0);
  const int first = h0 + warp * kPerWarp + lane / (D / 8);
  const __nv_bfloat16* in = src.p + (long long)row * src.ts + (long long)first * src.hs;
  uint4 v[kPass];
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (first + i * step < src.heads) v[i] = hl.read(in);
    in += step * src.hs;
  }
  float4 c, s;
  hl.angles(nr, max(pos, 0), c, s, err);
  float w[8];
  load_weight<D>(weight, hl, w);
  __nv_bfloat16* out = dst.p + (long long)row * dst.ts + (long long)first * dst.hs;
  if (pos < 0) {  // a padding row: zeros
    const float zero[8] = {};
    for (int h = first; h < min(src.heads, first + kPass * step); h += step, out += step * dst.hs) hl.write(out, zero);
    return;
  }
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    float x[8];
    unpack8(v[i], x);
    if (weight) head_norm<D>(x, w, nr.eps);
    hl.rotate(x, c, s);
    if (first + i * step < src.heads) hl.write(out, x);
    out += step * dst.hs;
  }
}

// Blocks y < q_chunks take query heads, the others key heads.
template <int D, int kPass>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x, y = blockIdx.y, pos = p.positions[row];
  if (y < p.q_chunks)
    rope_row<D, kPass>(p.q, p.qo, p.nr.q_weight, p.nr, row, pos, y * p.heads_per_block, p.err);
  else
    rope_row<D, kPass>(p.k, p.ko, p.nr.k_weight, p.nr, row, pos, (y - p.q_chunks) * p.heads_per_block, p.err);
}

// ---------------------------------------------------------------------- append
constexpr int kAppendThreads = 256;

struct AppendParams {
  KvHeads q, k, v, qo;
  KvCacheRef cache;
  KvBatch batch;
  NormRope nr;
  unsigned* err;
  int q_blocks;         // blocks that take query rows: rows * q_chunks
  int q_chunks;         // blocks a query row
  int heads_per_block;  // query heads of such a block
};

// The sequence of row `row` (-1: none), found by each warp in one pass over
// the row offsets.
__device__ __forceinline__ int find_row(const KvBatch& bt, int row) {
  if (!bt.q_start) return row;
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < bt.batch; b0 += 32) {
    const int b = b0 + lane;
    const bool here = b < bt.batch && bt.q_start[b] <= row && row < bt.q_start[b + 1];
    const unsigned any = __ballot_sync(0xffffffffu, here);
    if (any) return b0 + __ffs(any) - 1;
  }
  return -1;
}

// The page that the call's slot-th page write goes to: sequence and block of
// its table.  Pages are numbered by sequence, then by position; the block's
// threads scan the counts.  False past the last one.
__device__ __forceinline__ bool find_page(const KvBatch& bt, int page_shift, int slot, int* scratch, int* seq,
                                          int* block, unsigned* err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int* found = scratch + warps;
  if (threadIdx.x == 0) found[0] = -1;
  int base = 0;
  for (int b0 = 0; b0 < bt.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int count = 0, first = 0;
    if (b < bt.batch) {
      const KvSeq s = kv_seq(bt, page_shift, b, err);
      const int p0 = max(s.len - s.n, 0);
      if (s.n > 0 && s.len > p0) {
        first = p0 >> page_shift;
        count = ((s.len - 1) >> page_shift) - first + 1;
      }
    }
    int sum = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    __syncthreads();  // scratch of the round before is read
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    int before = base, total = 0;
    for (int w = 0; w < warps; ++w) {
      before += w < warp ? scratch[w] : 0;
      total += scratch[w];
    }
    const int at = slot - (before + sum - count);
    if (at >= 0 && at < count) {
      found[0] = b;
      found[1] = first + at;
    }
    base += total;
  }
  __syncthreads();
  *seq = found[0];
  *block = found[1];
  return found[0] >= 0;
}

// kPass: 256-thread passes over a page's new tokens (8 elements a thread);
// kQPass: passes of the query blocks over a row's heads.
template <int D, int kPass, int kQPass>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
  __shared__ int scratch[kAppendThreads / 32 + 2];
  pdl_launch_dependents();
  pdl_wait();
  if ((int)blockIdx.x < p.q_blocks) {
    const int row = (int)blockIdx.x / p.q_chunks, h0 = ((int)blockIdx.x % p.q_chunks) * p.heads_per_block;
    const int b = find_row(p.batch, row);
    if (b < 0) return;  // a row of no sequence
    const KvSeq s = kv_seq(p.batch, p.cache.page_shift, b, p.err);
    rope_row<D, kQPass>(p.q, p.qo, p.nr.q_weight, p.nr, row, s.len - s.n + row - s.row0, h0, p.err);
    return;
  }
  // ------------------------------------------------- one page's K or V of a head
  const int item = (int)blockIdx.x - p.q_blocks;
  const bool is_v = (item & 1) != 0;
  const int h = (item >> 1) % p.cache.heads, slot = (item >> 1) / p.cache.heads;
  int b, block;
  if (!find_page(p.batch, p.cache.page_shift, slot, scratch, &b, &block, p.err)) return;
  const int page = kv_page(p.batch, p.cache.num_pages, b, block, p.err);
  if (page < 0) return;
  const KvSeq s = kv_seq(p.batch, p.cache.page_shift, b, nullptr);
  const int page_size = 1 << p.cache.page_shift, page0 = block << p.cache.page_shift;
  const int first = s.len - s.n;                  // position of row s.row0; rows below 0 are padding
  const int t0 = max(max(first, 0), page0);       // the call's positions in this page
  const int t1 = min(s.len, page0 + page_size);
  const long long at = (long long)page * p.cache.page_stride + (long long)h * p.cache.head_stride;
  uint8_t* codes = (is_v ? p.cache.v : p.cache.k) + at;
  float* scale = (is_v ? p.cache.v_scale : p.cache.k_scale) + (long long)page * p.cache.scale_stride + h;
  const bool joined = t0 > page0;  // earlier positions keep their place under a common scale
  const int e_old = joined ? (int)((__float_as_uint(*scale) >> 23) & 0xFF) - 127 : kKvExpMin;

  constexpr int kLanes = D / 8, kTok = kAppendThreads / kLanes;  // tokens a pass
  const int lane = threadIdx.x & 31, tok = threadIdx.x / kLanes;
  const KvHeads& src = is_v ? p.v : p.k;
  const bool norm = !is_v && p.nr.k_weight;
  const HeadLane<D> hl(lane, is_v ? 0 : p.nr.rot, p.nr.interleaved != 0);
  uint4 v[kPass];
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int t = t0 + i * kTok + tok;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t < t1) v[i] = hl.read(src.p + (long long)(s.row0 + t - first) * src.ts + (long long)h * src.hs);
  }
  float w[8], x[kPass][8];
  load_weight<D>(norm ? p.nr.k_weight : nullptr, hl, w);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    if (t0 + i * kTok >= t1) break;  // no token of this pass in the block
    unpack8(v[i], x[i]);
    if (!is_v) {
      float4 cs, sn;
      hl.angles(p.nr, min(t0 + i * kTok + tok, t1 - 1), cs, sn, p.err);
      if (norm) head_norm<D>(x[i], w, p.nr.eps);
      hl.rotate(x[i], cs, sn);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(x[i][j]);
      if (a <= 3.402823466e38f) amax = fmaxf(amax, a);  // infinities and NaN do not count
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  __syncthreads();  // scratch is free
  if (lane == 0) scratch[threadIdx.x >> 5] = __float_as_int(amax);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, __int_as_float(scratch[i]));
  const int e = max(kv_scale_exp(amax), min(max(e_old, kKvExpMin), kKvExpMax));
  if (joined && e > e_old) {  // earlier codes to the larger scale
    const float f = kv_exp2i(e_old - e);
    for (int i = threadIdx.x; i < (t0 - page0) * (D / 16); i += kAppendThreads) {
      uint4* c = reinterpret_cast<uint4*>(codes + (long long)(i / (D / 16)) * p.cache.token_stride + i % (D / 16) * 16);
      uint4 v = *c;
      uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a0, a1, a2, a3;
        from_e4m3x4(u[j], a0, a1, a2, a3);
        u[j] = to_e4m3x4(a0 * f, a1 * f, a2 * f, a3 * f);
      }
      *c = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
  const float inv = kv_exp2i(-e);
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int t = t0 + i * kTok + tok;
    if (t < t1) {
      uint8_t* c = codes + (long long)(t - page0) * p.cache.token_stride;
      *reinterpret_cast<uint32_t*>(c + hl.o0) = to_e4m3x4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
      *reinterpret_cast<uint32_t*>(c + hl.o1) = to_e4m3x4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv);
    }
  }
  if (threadIdx.x == 0) *scale = kv_exp2i(e);
}

}  // namespace sgr
