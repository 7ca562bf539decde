// sgr_kv_attn.cuh -- attention of new tokens over the paged E4M3 cache
// (sgr_attention.h):  o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t).
#pragma once

#include "sgr_kv_append.cuh"

namespace sgr {

constexpr int kAttnThreads = 128;

struct AttnParams {
  KvHeads q, out;
  KvCacheRef cache;
  KvBatch batch;
  float scale_log2;  // scale * log2(e)
  int window;
  unsigned* err;
};

// One block per row and query head; each warp takes every fourth position
// with its own running maximum, sum and output, joined at the end.
template <int D>
__global__ void __launch_bounds__(kAttnThreads) kv_attn_kernel(const AttnParams p) {
  constexpr int kE = D / 32, kWarps = kAttnThreads / 32;
  __shared__ int found;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x, h = blockIdx.y, hk = h / (p.q.heads / p.cache.heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = find_row(p.batch, row, &found);
  if (b < 0) return;
  const KvSeq s = kv_seq(p.batch, p.cache.page_shift, b, p.err);
  const int pos = s.len - s.n + row - s.row0;
  const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  float q[kE], o[kE], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < kE; ++j) {
    q[j] = __bfloat162float(p.q.p[(long long)row * p.q.ts + (long long)h * p.q.hs + lane * kE + j]) * p.scale_log2;
    o[j] = 0.f;
  }
  for (int t = lo + warp; t <= pos; t += kWarps) {
    const int page = kv_page(p.batch, p.cache.num_pages, b, t >> p.cache.page_shift, p.err);
    if (page < 0) continue;
    const long long at = (long long)page * p.cache.page_stride + (long long)hk * p.cache.head_stride +
                         (long long)(t & ((1 << p.cache.page_shift) - 1)) * p.cache.token_stride + lane * kE;
    const long long sc = (long long)page * p.cache.scale_stride + hk;
    uint32_t kc, vc;
    if (kE == 4) {
      kc = *reinterpret_cast<const uint32_t*>(p.cache.k + at);
      vc = *reinterpret_cast<const uint32_t*>(p.cache.v + at);
    } else {
      kc = *reinterpret_cast<const uint16_t*>(p.cache.k + at);
      vc = *reinterpret_cast<const uint16_t*>(p.cache.v + at);
    }
    float kf[4], vf[4];
    from_e4m3x4(kc, kf[0], kf[1], kf[2], kf[3]);
    from_e4m3x4(vc, vf[0], vf[1], vf[2], vf[3]);
    float d = 0.f;
#pragma unroll
    for (int j = 0; j < kE; ++j) d = fmaf(q[j], kf[j], d);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
    d *= p.cache.k_scale[sc];
    const float mn = fmaxf(m, d), a = exp2f(m - mn), w = exp2f(d - mn), wv = w * p.cache.v_scale[sc];
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int j = 0; j < kE; ++j) o[j] = o[j] * a + wv * vf[j];
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int j = 0; j < kE; ++j) so[warp][lane * kE + j] = o[j];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kAttnThreads) {
    float mm = sm[0], ll = 0.f, oo = 0.f;
    for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, sm[w]);
    for (int w = 0; w < kWarps; ++w)
      if (sm[w] > -INFINITY) {
        const float a = exp2f(sm[w] - mm);
        ll += sl[w] * a;
        oo += so[w][d] * a;
      } else if (sl[w] != 0.f) {  // only NaN was seen
        ll += sl[w], oo += so[w][d];
      }
    p.out.p[(long long)row * p.out.ts + (long long)h * p.out.hs + d] = __float2bfloat16(ll == 0.f ? 0.f : oo / ll);
  }
}

}  // namespace sgr
