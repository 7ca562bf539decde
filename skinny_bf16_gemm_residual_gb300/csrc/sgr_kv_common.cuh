// sgr_kv_common.cuh -- device side of the structures of sgr_attention.h: the
// sequences of a call, heads of rows, and the norm + rotation of one head.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sgr_ptx.cuh"

namespace sgr {

constexpr int kKvExpMin = -64, kKvExpMax = 64;  // exponents of the page scales

struct KvHeads {
  __nv_bfloat16* p;
  long long ts, hs;  // token and head stride, elements
  int heads;
};

struct KvBatch {
  const int* table;
  const int* seq_len;
  const int* q_start;  // NULL: row b belongs to sequence b
  long long table_stride;
  int batch, max_pages, tokens;
};

struct KvCacheRef {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  long long page_stride, head_stride, token_stride, scale_stride;
  int num_pages, page_shift, heads;
};

// Rows and length of a sequence, brought into range (device data is the
// caller's; what does not fit is recorded and never followed).
struct KvSeq {
  int row0, n, len;
};

__device__ __forceinline__ KvSeq kv_seq(const KvBatch& bt, int page_shift, int b, unsigned* err) {
  KvSeq s;
  bool bad = false;
  s.len = bt.seq_len[b];
  if (bt.q_start) {
    const int r0 = bt.q_start[b], r1 = bt.q_start[b + 1];
    s.row0 = min(max(r0, 0), bt.tokens);
    const int e = min(max(r1, s.row0), bt.tokens);
    bad = s.row0 != r0 || e != r1;
    s.n = e - s.row0;
  } else {
    s.row0 = b;
    s.n = 1;
  }
  const long long room = (long long)bt.max_pages << page_shift;
  if (s.len < 0 || s.len > room) {
    bad = true;
    s.len = s.len < 0 ? 0 : (int)room;
  }
  if (bad) report_error(err, kErrIndex);
  return s;
}

// The page of a sequence's block, or -1 (recorded) when the table names none.
__device__ __forceinline__ int kv_page(const KvBatch& bt, int num_pages, int b, int block, unsigned* err) {
  const int p = bt.table[(long long)b * bt.table_stride + block];
  if (p >= 0 && p < num_pages) return p;
  report_error(err, kErrIndex);
  return -1;
}

// ------------------------------------------------------------ norm + rotation
struct NormRope {
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  const float* table;
  float eps;
  int table_rows, rot, interleaved;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  x[0] = bf16lo(v.x), x[1] = bf16hi(v.x), x[2] = bf16lo(v.y), x[3] = bf16hi(v.y);
  x[4] = bf16lo(v.z), x[5] = bf16hi(v.z), x[6] = bf16lo(v.w), x[7] = bf16hi(v.w);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A head of D elements is held by D / 8 neighbouring lanes, each with two runs
// of four elements, at o0 and o1, chosen so that a lane holds both elements
// of its four pairs: the same place of the two halves of the rotated part, or
// eight consecutive elements (interleaved pairs, elements past rot, no
// rotation).
template <int D>
struct HeadLane {
  int o0, o1;
  bool turns, split;  // whether the lane's elements are rotated, and as (run, run) pairs

  __device__ __forceinline__ HeadLane(int lane, int rot, bool interleaved) {
    const int l = lane % (D / 8);
    turns = 8 * l < rot;
    split = turns && !interleaved;
    o0 = split ? 4 * l : 8 * l;
    o1 = split ? rot / 2 + 4 * l : 8 * l + 4;
  }

  __device__ __forceinline__ uint4 read(const __nv_bfloat16* head) const {
    const uint2 a = *reinterpret_cast<const uint2*>(head + o0), b = *reinterpret_cast<const uint2*>(head + o1);
    return make_uint4(a.x, a.y, b.x, b.y);
  }

  __device__ __forceinline__ void write(__nv_bfloat16* head, const float (&x)[8]) const {
    *reinterpret_cast<uint2*>(head + o0) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    *reinterpret_cast<uint2*>(head + o1) = make_uint2(pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }

  // Cosines and sines of the lane's four pairs at a position.
  __device__ __forceinline__ void angles(const NormRope& nr, int pos, float4& c, float4& s, unsigned* err) const {
    c = s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!turns) return;
    if (pos >= nr.table_rows) {
      report_error(err, kErrIndex);
      pos = nr.table_rows - 1;
    }
    const float* row = nr.table + (long long)pos * nr.rot + (split ? o0 : o0 / 2);
    c = *reinterpret_cast<const float4*>(row);
    s = *reinterpret_cast<const float4*>(row + nr.rot / 2);
  }

  __device__ __forceinline__ void rotate(float (&x)[8], const float4& c, const float4& s) const {
    if (!turns) return;  // (and an infinity times a zero sine is not zero)
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
    if (split) {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn(x[j], x[4 + j], cc[j], ss[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn(x[2 * j], x[2 * j + 1], cc[j], ss[j]);
    }
  }

  static __device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float na = a * c - b * s, nb = b * c + a * s;
    a = na, b = nb;
  }
};

// The lane's 8 norm weights; ones where there are none.
template <int D>
__device__ __forceinline__ void load_weight(const __nv_bfloat16* w, const HeadLane<D>& hl, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = 1.f;
  if (w) unpack8(hl.read(w), x);
}

// RMS norm of the heads that the warp's lane groups hold (all lanes take part).
template <int D>
__device__ __forceinline__ void head_norm(float (&x)[8], const float (&w)[8], float eps) {
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float r = rsqrtf(fmaf(sum, 1.0f / D, eps));
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
}

}  // namespace sgr
