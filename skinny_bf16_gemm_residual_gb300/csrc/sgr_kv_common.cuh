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

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// A head of D elements is held by D / 8 neighbouring lanes, 8 consecutive
// elements each.  Element j of a lane becomes x_j c_j + partner_j s_j, its
// partner being the other of its pair: x_{j^1} of the same lane
// (interleaved), or element j of the lane rot/16 lanes up or down.  Lanes of
// elements past rot keep theirs (an infinity times a zero sine is not zero).
template <int D>
struct RopeLane {
  float c[8], s[8];
  int partner;  // lane of the warp that holds the other halves (not interleaved)
  bool turns;   // whether this lane's elements are rotated

  __device__ __forceinline__ void load(const NormRope& nr, int pos, int lane, unsigned* err) {
    const int l = lane % (D / 8), half = nr.rot / 2;
    partner = lane;
    turns = 8 * l < nr.rot;  // rot = 0: no rotation
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = s[j] = 0.f;
    if (!turns) return;
    if (pos >= nr.table_rows) {
      report_error(err, kErrIndex);
      pos = nr.table_rows - 1;
    }
    const float* row = nr.table + (long long)pos * nr.rot;
    if (nr.interleaved) {
      const float4 cv = *reinterpret_cast<const float4*>(row + 4 * l);
      const float4 sv = *reinterpret_cast<const float4*>(row + half + 4 * l);
      const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[2 * j] = c[2 * j + 1] = cc[j];
        s[2 * j] = -ss[j];
        s[2 * j + 1] = ss[j];
      }
    } else {
      const bool second = 8 * l >= half;
      const int i = second ? 8 * l - half : 8 * l;
      partner = second ? lane - half / 8 : lane + half / 8;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 cv = *reinterpret_cast<const float4*>(row + i + 4 * q);
        const float4 sv = *reinterpret_cast<const float4*>(row + half + i + 4 * q);
        c[4 * q] = cv.x, c[4 * q + 1] = cv.y, c[4 * q + 2] = cv.z, c[4 * q + 3] = cv.w;
        s[4 * q] = sv.x, s[4 * q + 1] = sv.y, s[4 * q + 2] = sv.z, s[4 * q + 3] = sv.w;
      }
      if (!second) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = -s[j];
      }
    }
  }

  // Rotation of the heads that the warp's lane groups hold (all lanes take part).
  __device__ __forceinline__ void rotate(float (&x)[8], bool interleaved) const {
    float y[8];
    if (interleaved) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], partner);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = turns ? fmaf(y[j], s[j], x[j] * c[j]) : x[j];
  }
};

// RMS norm of the heads that the warp's lane groups hold, where `norm` (all
// lanes take part).
template <int D>
__device__ __forceinline__ void head_norm(float (&x)[8], const float (&w)[8], bool norm, float eps) {
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float r = norm ? 1.0f / sqrtf(sum * (1.0f / D) + eps) : 1.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
}

// A lane's 8 norm weights; ones where there are none.
__device__ __forceinline__ void load_weight(const __nv_bfloat16* w, int lane_in_head, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = 1.f;
  if (w) unpack8(*reinterpret_cast<const uint4*>(w + 8 * lane_in_head), x);
}

}  // namespace sgr
