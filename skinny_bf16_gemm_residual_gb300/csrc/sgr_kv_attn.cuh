// sgr_kv_attn.cuh -- attention of new tokens over the paged E4M3 cache
// (sgr_attention.h):
//
//     o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q.k_t)
//
// Per row tile (up to NT query rows that share a key/value head: the head's
// query group, times the new tokens) and 128-token tile of the cache:
//
//     S^T [128 tokens, NT] = K Q^T      codes of K as they are in the cache
//     P^T = 2^(S' - m)                  one thread per token
//     O^T [D, NT]          = V^T P^T    codes of V as they are, read M-major
//
// Both products run on the FP8 tensor core (tcgen05.mma kind::f8f6f4) with
// the cache's codes as the 128-row operand straight from TMA, so that nothing
// is converted per cached element.  The small operands are brought into E4M3
// as two parts b = hi + lo / 32, each row (or tile) scaled by a power of two
// that puts its largest magnitude in [128, 256]: hi = e4m3(b),
// lo = e4m3(32 (b - hi)).  That holds 8 significant bits (all of a BF16
// query) down to 2^-14 of the largest and an absolute 2^-22 of it below.  hi
// and lo rows sit side by side in the operand (2 NT columns of the
// accumulator) and are added in FP32.
//
// Softmax: the maximum m of a tile's column is rounded up to a whole number,
// so every rescaling is by a power of two: exact, without the exponential
// unit, and P uses E4M3's whole range in every tile however far the running
// maximum lies above it.  The product of a tile is read back and accumulated
// in registers (thread d holds o[.][d]), O = O 2^(M-M') + O_tile 2^(m-M'), so
// no accumulator in tensor memory is ever rescaled.  A page's key scale
// multiplies the score; its value scale 2^e is added to the exponent of P and
// taken out of the sum of weights again.
//
// Work split: every CTA takes the same number of (row tile, 128-token tile)
// units of all sequences and heads, in order, whatever the lengths; a row
// tile that spans CTAs leaves partial sums (o, M, l) in the workspace and a
// second kernel joins them in order (the same bits on every run).
//
// Bound: the cache bytes, 2 D a token and key/value head, each read once per
// row tile.
//
// Roles (256 threads, two CTAs an SM): warps 0-3 softmax (thread = token,
// then = element d), warp 4 walks the work, loads pages by TMA and hands out
// segments, warp 5 issues the MMAs, warps 6-7 bring the next segment's
// queries into the operand.
#pragma once

#include <cuda.h>

#include "sgr_internal.h"
#include "sgr_kv_append.cuh"

namespace sgr {

constexpr int kAttnThreads = 256;
constexpr int kAttnTile = 128;  // tokens
constexpr int kAttnQueue = 8;   // segments handed out ahead

// A run of tiles [ta, tb) of one row tile, the unit that the roles work by.
enum : int { kSegStart = 1, kSegEnd = 2, kSegStop = 4 };
struct AttnSeg {
  int kind;
  int h, row0, r0, nrows;  // key/value head; the sequence's first row; rows r0 .. r0+nrows-1 of its n * group
  int first;               // position of the sequence's first row
  int ta, tb;
  int tlo, thi;  // positions that some row of the tile sees
  int slot;      // of its partial sums
  int pad;
};

// A partial sum's owner, for the kernel that joins them.
struct AttnPiece {
  int valid, last;
  int h, row0, r0, nrows;
  int pad[2];
};

struct AttnParams {
  KvHeads q, out;
  KvCacheRef cache;
  KvBatch batch;
  float scale_log2;  // scale * log2(e)
  int window;        // INT_MAX: none
  int group;         // query heads a key/value head
  int reuse;         // row tiles of a sequence share the cache's bytes
  unsigned* err;
  float* part_o;  // [2 grid][NT][D]
  float2* part_ml;  // [2 grid][NT]  maximum, sum
  AttnPiece* pieces;  // [2 grid]
};

template <int D, int NT>
struct AttnShape {
  static constexpr int kCols = 2 * NT;  // hi and lo rows of the small operands
  static constexpr int kTileBytes = kAttnTile * D;
  static constexpr int kStageBytes = 2 * kTileBytes;  // V, then K
  // As deep as two CTAs an SM allow.
  static constexpr int kStages = D == 128 ? (NT <= 16 ? 3 : 2) : (NT <= 16 ? 6 : 4);
  static constexpr int kPBytes = kCols * kAttnTile;
  static constexpr int kQBytes = kCols * D;
  static constexpr int kTmemCols = 4 * kCols < 32 ? 32 : 4 * kCols;  // S and O, two each
};

template <int NT>
struct AttnCtl {
  uint64_t kfull[6], vfull[6], empty[6];
  uint64_t sfull[2], sempty[2], ofull[2], oempty[2], qfull[2], qempty[2], pfull, drain;
  uint64_t segfull[kAttnQueue], segempty[kAttnQueue];
  uint32_t tmem;
  int abort;
  int go[2];
  int start_b;
  unsigned nan_tokens[4];
  long long start_off, units;
  long long scan[kAttnThreads / 32];
  AttnSeg seg[kAttnQueue];
  float kscale[6][8], vexp[6][8];  // of a stage's pages
  int flags[6];                    // 1: some token is not live, 2: rows see different tokens
  alignas(16) float qf[2][NT];     // score factor of a row
  int qpos[2][NT];                 // last position that a row sees
  long long qout[2][NT];           // its place in the output
  alignas(16) float wmax[2][4][NT], wsum[4][NT];
  alignas(16) float m[4][NT], alpha[4][2][NT], beta[4][2][NT];  // each softmax warp's own copy
};

template <int D, int NT>
constexpr int attn_ctl_bytes() {
  return (int)((sizeof(AttnCtl<NT>) + 1023) / 1024 * 1024);
}

template <int D, int NT>
constexpr int attn_smem_bytes() {
  using S = AttnShape<D, NT>;
  return 1024 + attn_ctl_bytes<D, NT>() + S::kStages * S::kStageBytes + S::kPBytes + 2 * S::kQBytes;
}

// Row tile j of a sequence: its rows, the positions they see, its units (a
// row tile that sees nothing is one unit: its zeros).
struct AttnItem {
  int r0, nrows, tlo, thi, ta, tb;
  __device__ __forceinline__ int units() const { return tb > ta ? tb - ta : 1; }
};

template <int NT>
__device__ __forceinline__ AttnItem attn_item(const KvSeq& s, int group, int window, int j) {
  AttnItem it;
  it.r0 = j * NT;
  it.nrows = min(NT, s.n * group - it.r0);
  const int first = s.len - s.n, p0 = first + it.r0 / group;
  it.thi = max(first + (it.r0 + it.nrows - 1) / group + 1, 0);
  it.tlo = window > p0 ? 0 : p0 - window + 1;
  it.ta = it.thi > 0 ? it.tlo / kAttnTile : 0;
  it.tb = (it.thi + kAttnTile - 1) / kAttnTile;
  return it;
}

template <int NT>
__device__ __forceinline__ long long attn_seq_units(const KvSeq& s, int group, int window) {
  const int nt = (s.n * group + NT - 1) / NT;
  long long u = 0;
  for (int j = 0; j < nt; ++j) u += attn_item<NT>(s, group, window, j).units();
  return u;
}

// 2^d for whole d <= 0 (0 from -127 down), on the integer unit.
__device__ __forceinline__ float exp2_whole(float d) {
  return __int_as_float((__float_as_int(fmaxf(d, -127.f) + 12582912.f) << 23) + 0x3f800000);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void sts8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

constexpr float kLoScale = 1.f / 32.f;

// Two values in [0, 256] -> their hi codes (bytes 0, 1) and lo codes (bytes 2,
// 3).  (FP16 holds b to 11 bits, b - hi exactly.)
__device__ __forceinline__ uint32_t split2(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b16 h, l;\n\t.reg .b32 x, y;\n\t"
      "cvt.rn.f16x2.f32 x, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 h, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, h;\n\t"
      "sub.rn.f16x2 x, x, y;\n\t"
      "mul.rn.f16x2 x, x, %3;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 l, x;\n\t"
      "mov.b32 %0, {h, l};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "r"(0x50005000u));  // 0x5000 = 32
  return r;
}

template <int NT>
__device__ __forceinline__ void tmem_ld_sum(uint32_t taddr, float (&x)[NT]) {
  // columns [0, NT) (hi) plus columns [NT, 2 NT) (lo) / 32
  if constexpr (NT == 8) {
    float v[16];
    tmem_ld16(taddr, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = fmaf(v[8 + q], kLoScale, v[q]);
  } else {
#pragma unroll
    for (int c = 0; c < NT; c += 16) {
      float v[16], w[16];
      tmem_ld16(taddr + c, v);
      tmem_ld16(taddr + NT + c, w);
#pragma unroll
      for (int q = 0; q < 16; ++q) x[c + q] = fmaf(w[q], kLoScale, v[q]);
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, 2)
    kv_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
  using Sh = AttnShape<D, NT>;
  constexpr int S = Sh::kStages, kCols = Sh::kCols;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  AttnCtl<NT>& c = *reinterpret_cast<AttnCtl<NT>*>(smem_raw + (base - raw));
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
      mbar_init(smem_u32(&c.sfull[i]), 1);
      mbar_init(smem_u32(&c.sempty[i]), 4);
      mbar_init(smem_u32(&c.ofull[i]), 1);
      mbar_init(smem_u32(&c.oempty[i]), 4);
      mbar_init(smem_u32(&c.qfull[i]), 2);
      mbar_init(smem_u32(&c.qempty[i]), 5);  // the last MMA that reads it, the softmax warps
    }
    mbar_init(smem_u32(&c.pfull), 4);
    mbar_init(smem_u32(&c.drain), 1);
    for (int i = 0; i < kAttnQueue; ++i) {
      mbar_init(smem_u32(&c.segfull[i]), 1);
      mbar_init(smem_u32(&c.segempty[i]), 7);  // MMA, 4 softmax and 2 query warps
    }
    c.abort = 0;
    c.start_b = -1;
    fence_mbar_init();
  }
  if (warp == 5) {
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
  pdl_wait();

  // ------------------------------------------------ this CTA's share of the work
  const int ps = p.cache.page_shift, hk = p.cache.heads;
  long long mine = 0;
  for (int b = tid; b < p.batch.batch; b += kAttnThreads)
    mine += attn_seq_units<NT>(kv_seq(p.batch, ps, b, p.err), p.group, p.window);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) c.scan[warp] = mine;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kAttnThreads / 32; ++w) total += c.scan[w];
  total *= hk;
  // (with fewer units than CTAs the last ones have none, the others one each)
  const long long active = min(total, (long long)gridDim.x);
  const bool busy = blockIdx.x < active;
  const long long u0 = busy ? total * blockIdx.x / active : 0, u1 = busy ? total * (blockIdx.x + 1) / active : 0;
  {
    long long before = 0;  // units of the sequences before this round's
    for (int b0 = 0; b0 < p.batch.batch && u1 > u0; b0 += kAttnThreads) {
      const int b = b0 + tid;
      long long u = 0;
      if (b < p.batch.batch) u = hk * attn_seq_units<NT>(kv_seq(p.batch, ps, b, nullptr), p.group, p.window);
      long long sum = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      __syncthreads();
      if (lane == 31) c.scan[warp] = sum;
      __syncthreads();
      long long at = before + sum - u;
#pragma unroll
      for (int w = 0; w < kAttnThreads / 32; ++w) {
        at += w < warp ? c.scan[w] : 0;
        before += c.scan[w];
      }
      if (u0 >= at && u0 < at + u) {
        c.start_b = b;
        c.start_off = u0 - at;
      }
      if (before > u0) break;
    }
  }
  __syncthreads();

  if (warp == 4) {
    // ------------------------------------------------------- walk and TMA loads
    const uint64_t policy = p.reuse ? policy_evict_last() : policy_evict_first();
    int b = c.start_b, h = 0, j = 0, skip = 0, sq = 0, pieces = 0;
    long long left = b >= 0 ? u1 - u0 : 0;
    KvSeq s{0, 0, 0};
    AttnItem it{};
    bool ok = true;
    if (left > 0) {
      s = kv_seq(p.batch, ps, b, nullptr);
      const long long per = attn_seq_units<NT>(s, p.group, p.window);
      long long off = c.start_off;
      h = (int)(off / per);
      off -= h * per;
      it = attn_item<NT>(s, p.group, p.window, 0);
      while (off >= it.units()) {
        off -= it.units();
        it = attn_item<NT>(s, p.group, p.window, ++j);
      }
      skip = (int)off;
    }
    int t = 0, t_end = 0;  // tiles of the segment handed out last
    auto hand_out = [&](const AttnSeg& g) {
      const int qi = sq % kAttnQueue;
      if (ok && !mbar_wait_or_abort(smem_u32(&c.segempty[qi]), ((sq / kAttnQueue) & 1) ^ 1, abort_flag)) {
        if (!*abort_flag) report_error(p.err, kErrWaitEmpty);
        *abort_flag = 1;
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) {
        c.seg[qi] = g;
        mbar_arrive(smem_u32(&c.segfull[qi]));
      }
      ++sq;
    };
    // The next tile of this CTA's share; hands out the segments it enters.
    struct Tile {
      int tile, h, flags, page;  // page: this lane's, -1 = none
      float ks, vs;
    };
    AttnItem cur{};
    int cur_h = 0, cur_b = 0, cur_p0 = 0, cur_p1 = 0;
    auto next_tile = [&](Tile& x) -> bool {
      while (t == t_end) {
        if (left <= 0 || !ok) return false;
        const int nt = (s.n * p.group + NT - 1) / NT;
        if (j >= nt || s.n == 0) {
          j = 0;
          if (s.n == 0 || ++h == hk) {
            h = 0;
            do {
              if (++b >= p.batch.batch) return false;
              s = kv_seq(p.batch, ps, b, nullptr);
            } while (s.n == 0);
          }
          it = attn_item<NT>(s, p.group, p.window, 0);
        }
        const int units = it.units(), take = (int)min(left, (long long)(units - skip));
        left -= take;
        if (it.tb <= it.ta) {  // rows that see nothing: zeros
          for (int e = lane; e < it.nrows * (D / 8); e += 32) {
            const int r = it.r0 + e / (D / 8);
            *reinterpret_cast<uint4*>(p.out.p + (long long)(s.row0 + r / p.group) * p.out.ts +
                                      (long long)(h * p.group + r % p.group) * p.out.hs + e % (D / 8) * 8) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          it = attn_item<NT>(s, p.group, p.window, ++j);
          continue;
        }
        AttnSeg g;
        g.kind = (skip == 0 ? kSegStart : 0) | (skip + take == units ? kSegEnd : 0);
        g.h = h;
        g.row0 = s.row0;
        g.r0 = it.r0;
        g.nrows = it.nrows;
        g.first = s.len - s.n;
        g.ta = it.ta + skip;
        g.tb = g.ta + take;
        g.tlo = it.tlo;
        g.thi = it.thi;
        g.slot = 2 * (int)blockIdx.x + (skip == 0 ? 1 : 0);
        g.pad = 0;
        if (lane == 0 && (g.kind & (kSegStart | kSegEnd)) != (kSegStart | kSegEnd)) {
          AttnPiece pc = {1, (g.kind & kSegEnd) ? 1 : 0, h, s.row0, it.r0, it.nrows, {0, 0}};
          p.pieces[g.slot] = pc;
        }
        if ((g.kind & (kSegStart | kSegEnd)) != (kSegStart | kSegEnd)) pieces |= 1 << (g.slot & 1);
        hand_out(g);
        if (!ok) return false;
        t = g.ta;
        t_end = g.tb;
        cur = it;
        cur_h = h;
        cur_b = b;
        cur_p0 = g.first + it.r0 / p.group;
        cur_p1 = it.thi - 1;
        skip = 0;
        if (g.kind & kSegEnd) it = attn_item<NT>(s, p.group, p.window, ++j);
      }
      const int x0 = t * kAttnTile, x1 = x0 + kAttnTile;
      x.tile = t++;
      x.h = cur_h;
      x.flags = (x0 < cur.tlo || x1 > cur.thi) ? 1 : 0;
      if (min(x1, cur.thi) - 1 > max(cur_p0, -1) || max(x0, cur.tlo) < (long long)cur_p1 - p.window + 1) x.flags |= 2;
      // This lane's page of the tile, where some row sees a position of it.
      const int block = (x0 >> ps) + lane, at = block << ps;
      x.page = -1;
      if (lane < (kAttnTile >> ps) && at < cur.thi && at + (1 << ps) > cur.tlo)
        x.page = kv_page(p.batch, p.cache.num_pages, cur_b, block, p.err);
      return true;
    };
    auto load_scales = [&](Tile& x) {
      x.ks = x.vs = 0.f;
      if (x.page >= 0) {
        const long long at = (long long)x.page * p.cache.scale_stride + x.h;
        x.ks = p.cache.k_scale[at];
        x.vs = p.cache.v_scale[at];
      }
    };
    // Two tiles ahead of the copies: table entries, then (dependent) scales.
    Tile a{}, n1{}, n2{};
    bool has_a = next_tile(a), has_1 = has_a && next_tile(n1);
    if (has_a) load_scales(a);
    int i = 0;
    while (has_a && ok) {
      const bool has_2 = has_1 && next_tile(n2);
      if (has_1) load_scales(n1);
      const int slot = i % S;
      if (i >= S && !mbar_wait_or_abort(smem_u32(&c.empty[slot]), ((i / S) & 1) ^ 1, abort_flag)) {
        if (!*abort_flag) report_error(p.err, kErrWaitEmpty);
        *abort_flag = 1;
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int per_tile = kAttnTile >> ps;
      const unsigned live = __ballot_sync(0xffffffffu, a.page >= 0);
      if (lane < per_tile) {
        c.kscale[slot][lane] = a.ks;
        // (an exponent of -inf marks a page that is not there)
        c.vexp[slot][lane] = a.page >= 0 ? (float)((int)((__float_as_uint(a.vs) >> 23) & 0xFF) - 127) : -INFINITY;
      }
      if (lane == 0) c.flags[slot] = a.flags | (__popc(live) < per_tile ? 1 : 0);
      __syncwarp();
      const uint32_t kb = smem_u32(&c.kfull[slot]), vb = smem_u32(&c.vfull[slot]);
      const uint32_t page_bytes = (uint32_t)D << ps;
      if (lane == 0) {
        mbar_arrive_expect_tx(kb, (uint32_t)__popc(live) * page_bytes);
        mbar_arrive_expect_tx(vb, (uint32_t)__popc(live) * page_bytes);
      }
      __syncwarp();
      if (a.page >= 0) {
        const uint32_t dst = ring + (uint32_t)slot * Sh::kStageBytes + (uint32_t)lane * page_bytes;
        tma_load_4d(dst + Sh::kTileBytes, &tmK, 0, 0, a.h, a.page, kb, policy);
        tma_load_4d(dst, &tmV, 0, 0, a.h, a.page, vb, policy);
      }
      ++i;
      a = n1;
      n1 = n2;
      has_a = has_1;
      has_1 = has_2;
    }
    AttnSeg stop{};
    stop.kind = kSegStop;
    hand_out(stop);
    if (lane < 2 && !(pieces >> lane & 1)) p.pieces[2 * blockIdx.x + lane].valid = 0;
    // Every copy that this warp issued lands before the CTA may exit.
    bool landed = true;
    for (int k = i > S ? i - S : 0; k < i && landed; ++k)
      landed = mbar_wait(smem_u32(&c.kfull[k % S]), (k / S) & 1) && mbar_wait(smem_u32(&c.vfull[k % S]), (k / S) & 1);
    if (!landed) report_error(p.err, kErrDrain);
  } else if (warp == 5) {
    // ------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_e4m3_f32(kAttnTile, kCols), idesc_o = idesc_s | (1u << 15);
      const uint32_t acc_o = tmem + 2 * kCols;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !mbar_wait_or_abort(smem_u32(bar), parity, abort_flag)) {
          if (!*abort_flag) report_error(p.err, kErrWaitFull);
          *abort_flag = 1;
          ok = false;
        }
      };
      // O of tile k = V^T P^T, once its weights are written.
      auto value_product = [&](int k) {
        const int slot = k % S;
        wait(&c.vfull[slot], (k / S) & 1);
        wait(&c.pfull, k & 1);
        wait(&c.oempty[k & 1], ((k >> 1) & 1) ^ 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t v = ring + (uint32_t)slot * Sh::kStageBytes;
        // D = 64: the upper half of the 128 rows reads the K tile behind V;
        // its rows of the accumulator are not used.
        const uint64_t vd = smem_desc_rows<D>(v, Sh::kTileBytes), pd = smem_desc_rows<128>(pbuf);
#pragma unroll
        for (int kk = 0; kk < kAttnTile / 32; ++kk)
          mma_e4m3(acc_o + (k & 1) * kCols, vd + (uint64_t)(kk * (32 * D >> 4)), pd + (uint64_t)(kk * 2), idesc_o, kk > 0);
        mma_commit(smem_u32(&c.ofull[k & 1]));
        mma_commit(smem_u32(&c.empty[slot]));
      };
      int i = 0, sq = 0, filled = 0;
      while (ok) {
        const int qi = sq % kAttnQueue;
        wait(&c.segfull[qi], (sq / kAttnQueue) & 1);
        if (!ok) break;
        const int kind = c.seg[qi].kind, ta = c.seg[qi].ta, tb = c.seg[qi].tb;
        mbar_arrive(smem_u32(&c.segempty[qi]));
        ++sq;
        if (kind & kSegStop) break;
        wait(&c.qfull[filled & 1], (filled >> 1) & 1);
        const uint64_t qd = smem_desc_rows<D>(qbuf + (filled & 1) * Sh::kQBytes);
        for (int t = ta; t < tb && ok; ++t, ++i) {
          const int slot = i % S;
          wait(&c.kfull[slot], (i / S) & 1);
          wait(&c.sempty[i & 1], ((i >> 1) & 1) ^ 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = smem_desc_rows<D>(ring + (uint32_t)slot * Sh::kStageBytes + Sh::kTileBytes);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_e4m3(tmem + (i & 1) * kCols, kd + (uint64_t)(kk * 2), qd + (uint64_t)(kk * 2), idesc_s, kk > 0);
          mma_commit(smem_u32(&c.sfull[i & 1]));
          if (t == tb - 1) mma_commit(smem_u32(&c.qempty[filled & 1]));
          if (i > 0) value_product(i - 1);
        }
        ++filled;
      }
      if (ok && i > 0) value_product(i - 1);
      mma_commit(smem_u32(&c.drain));
      if (!mbar_wait(smem_u32(&c.drain), 0)) report_error(p.err, kErrDrain);
    }
  } else if (warp >= 6) {
    // ----------------------------------------------------------- query operand
    constexpr int kLanes = D / 8, kRows = 64 / kLanes, kPass = NT / kRows > 0 ? NT / kRows : 1;
    const int qt = tid - 192, l = qt % kLanes;
    int sq = 0, filled = 0;
    while (true) {
      const int qi = sq % kAttnQueue;
      bool ok = true;
      if (lane == 0) ok = mbar_wait_sleepy_or_abort(smem_u32(&c.segfull[qi]), (sq / kAttnQueue) & 1, abort_flag);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      const AttnSeg g = c.seg[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.segempty[qi]));
      ++sq;
      if (g.kind & kSegStop) break;
      const int buf = filled & 1;
      uint4 v[kPass];
      long long out_at[kPass];
      int pos[kPass];
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        const int q = i * kRows + qt / kLanes, r = g.r0 + q;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        pos[i] = -1;  // a row that is none sees nothing
        out_at[i] = 0;
        if (q < g.nrows) {
          const int tok = r / p.group, head = g.h * p.group + r % p.group;
          pos[i] = g.first + tok;
          out_at[i] = (long long)(g.row0 + tok) * p.out.ts + (long long)head * p.out.hs;
          v[i] = *reinterpret_cast<const uint4*>(p.q.p + (long long)(g.row0 + tok) * p.q.ts + (long long)head * p.q.hs + 8 * l);
        }
      }
      if (lane == 0) ok = mbar_wait_sleepy_or_abort(smem_u32(&c.qempty[buf]), ((filled >> 1) & 1) ^ 1, abort_flag);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        const int q = i * kRows + qt / kLanes;
        uint32_t mag = 0;
        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) mag = max(mag, max(u[k] & 0x7FFFu, (u[k] >> 16) & 0x7FFFu));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, o));
        const int ex = (int)(mag >> 7);  // biased exponent of the row's largest magnitude
        int k = ex == 0 ? 126 : 134 - ex;
        k = min(max(k, -120), 126);
        const float sc = kv_exp2i(k);
        float x[8], h[8];
        unpack8(v[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= sc;
        const uint2 hi = make_uint2(to_e4m3x4(x[0], x[1], x[2], x[3]), to_e4m3x4(x[4], x[5], x[6], x[7]));
        from_e4m3x4(hi.x, h[0], h[1], h[2], h[3]);
        from_e4m3x4(hi.y, h[4], h[5], h[6], h[7]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (x[e] - h[e]) * 32.f;  // exact
        const uint2 lo = make_uint2(to_e4m3x4(x[0], x[1], x[2], x[3]), to_e4m3x4(x[4], x[5], x[6], x[7]));
        if (q < NT) {
          const uint32_t qb = qbuf + (uint32_t)(buf * Sh::kQBytes) + (uint32_t)((l & 1) * 8);
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qb + swizzled<D>(q, l >> 1)), "r"(hi.x), "r"(hi.y) : "memory");
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qb + swizzled<D>(NT + q, l >> 1)), "r"(lo.x), "r"(lo.y) : "memory");
          if (l == 0) {
            // a row with an infinity or NaN gets NaN
            c.qf[buf][q] = ex == 255 ? __int_as_float(0x7fffffff) : kv_exp2i(-k) * p.scale_log2;
            c.qpos[buf][q] = pos[i];
            c.qout[buf][q] = out_at[i];
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.qfull[buf]));
      ++filled;
    }
  } else {
    // ---------------------------------------------------------------- softmax
    // After a wait that ran out (abort) the waits fall through, so that all
    // four warps keep meeting at their barrier until the segments end.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar_wait_or_abort(smem_u32(bar), parity, abort_flag)) {
        if (!*abort_flag) report_error(p.err, kErrWaitMma);
        *abort_flag = 1;
      }
      __syncwarp();
    };
    const uint32_t lane_base = (uint32_t)warp << 21;  // tensor-memory lane 32 warp
    float o[NT], l[NT];
    float run = 0.f;  // running maximum of row `lane`
    unsigned nan_rows = 0;
    int i = 0, sq = 0, filled = 0;
    // O of tile k, read back and accumulated.
    auto accumulate = [&](int k) {
      wait(&c.ofull[k & 1], (k >> 1) & 1);
      tc_fence_after();
      float x[NT];
      tmem_ld_sum<NT>(tmem + lane_base + 2 * kCols + (k & 1) * kCols, x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.oempty[k & 1]));
#pragma unroll
      for (int q = 0; q < NT; ++q) o[q] = fmaf(x[q], c.beta[warp][k & 1][q], o[q] * c.alpha[warp][k & 1][q]);
    };
    while (true) {
      const int qi = sq % kAttnQueue;
      if (tid == 0)
        c.go[sq & 1] = mbar_wait_sleepy_or_abort(smem_u32(&c.segfull[qi]), (sq / kAttnQueue) & 1, abort_flag) ? 1 : 0;
      __syncwarp();
      named_bar_sync(1, 128);
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
      const int buf = filled & 1;
      wait(&c.qfull[buf], (filled >> 1) & 1);
#pragma unroll
      for (int q = 0; q < NT; ++q) o[q] = l[q] = 0.f;
      run = -3.0e38f;
      nan_rows = 0;
      for (int t = g.ta; t < g.tb; ++t, ++i) {
        const int slot = i % S, sb = i & 1;
        wait(&c.sfull[sb], (i >> 1) & 1);
        wait(&c.kfull[slot], (i / S) & 1);  // (orders this thread's reads of the page scales)
        tc_fence_after();
        float x[NT];
        tmem_ld_sum<NT>(tmem + lane_base + sb * kCols, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.sempty[sb]));
        const int pi = tid >> ps, flags = c.flags[slot], pos = t * kAttnTile + tid;
        const float ks = c.kscale[slot][pi], ve = c.vexp[slot][pi];
        const bool live = !(flags & 1) || (pos >= g.tlo && pos < g.thi && ve > -INFINITY);
#pragma unroll
        for (int q = 0; q < NT; ++q) x[q] = fmaf(x[q], ks * c.qf[buf][q], ve);
        if (flags & 2) {
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            const int last = c.qpos[buf][q];
            if (!(live && pos <= last && pos > last - p.window)) x[q] = -INFINITY;
          }
        } else if (!live) {
#pragma unroll
          for (int q = 0; q < NT; ++q) x[q] = -INFINITY;
        }
        // The tile's maximum of each row, rounded up; lane q keeps row q's.
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const float w = warp_max(x[q]);
          if (lane == q) top = w;
        }
        if (lane < NT) c.wmax[sb][warp][lane] = top;
        __syncwarp();
        named_bar_sync(1, 128);
        if (lane < NT) {
          top = fmaxf(fmaxf(c.wmax[sb][0][lane], c.wmax[sb][1][lane]), fmaxf(c.wmax[sb][2][lane], c.wmax[sb][3][lane]));
          const float m = fmaxf(ceilf(top), -3.0e38f), now = fmaxf(run, m);
          c.m[warp][lane] = m;
          c.alpha[warp][sb][lane] = exp2_whole(run - now);
          c.beta[warp][sb][lane] = exp2_whole(m - now);
          run = now;
        }
        __syncwarp();
        const float iv = live ? kv_exp2i(-(int)ve) : 0.f;  // the value scale does not count in the sum of weights
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          x[q] = ex2(x[q] - c.m[warp][q]);
          l[q] = fmaf(x[q] * iv, c.beta[warp][sb][q], l[q] * c.alpha[warp][sb][q]);
        }
        const bool joined = t > g.ta;
        if (joined) wait(&c.ofull[(i - 1) & 1], ((i - 1) >> 1) & 1);  // the weights before are read
        if (flags) {
          wait(&c.vfull[slot], (i / S) & 1);
          const uint32_t vt = ring + (uint32_t)slot * Sh::kStageBytes;
          // Values of tokens that no row sees must not reach the product
          // (0 x NaN): their codes become zeros.
          if (!live) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + (uint32_t)(tid * D + k * 16)), "r"(0u) : "memory");
          }
          if (flags & 2) {
            // A NaN value that some rows see and others do not: those that do
            // get their NaN below, and the code becomes zero.
            bool nan = false;
            if (live) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint4 u = lds128(vt + (uint32_t)(tid * D + k * 16));
                const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) nan |= (((w4[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
              }
            }
            const unsigned any = __ballot_sync(0xffffffffu, nan);
            if (lane == 0) c.nan_tokens[warp] = any;
            __syncwarp();
            named_bar_sync(1, 128);
            if ((c.nan_tokens[0] | c.nan_tokens[1] | c.nan_tokens[2] | c.nan_tokens[3]) != 0) {
              for (int k = 0; k < kAttnTile; ++k) {
                if (!(c.nan_tokens[k >> 5] >> (k & 31) & 1) || tid >= D) continue;
                const uint32_t at = vt + swizzled<D>(k, tid >> 4) + (tid & 15);
                if ((lds8(at) & 0x7F) != 0x7F) continue;
                for (int q = 0; q < NT; ++q) {
                  const int last = c.qpos[buf][q], kp = t * kAttnTile + k;
                  if (kp <= last && kp > last - p.window) nan_rows |= 1u << q;
                }
                sts8(at, 0);
              }
              __syncwarp();
              named_bar_sync(1, 128);  // nan_tokens is read
            }
          }
        }
        const uint32_t col = (uint32_t)(tid & 15), chunk = tid >> 4;
#pragma unroll
        for (int q = 0; q < NT; q += 2) {
          const uint32_t u = split2(x[q] * 256.f, x[q + 1] * 256.f);
          sts8(pbuf + swizzled<128>(q, chunk) + col, u);
          sts8(pbuf + swizzled<128>(q + 1, chunk) + col, u >> 8);
          sts8(pbuf + swizzled<128>(NT + q, chunk) + col, u >> 16);
          sts8(pbuf + swizzled<128>(NT + q + 1, chunk) + col, u >> 24);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.pfull));
        if (joined) accumulate(i - 1);
      }
      accumulate(i - 1);
      // ------------------------------------------------------- the segment's end
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        float w = l[q];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
        if (lane == 0) c.wsum[warp][q] = w;
      }
      __syncwarp();
      named_bar_sync(1, 128);
      const float nan_f = __int_as_float(0x7fffffff);
      const bool whole = (g.kind & (kSegStart | kSegEnd)) == (kSegStart | kSegEnd);
      if (tid < D) {
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          if (q < g.nrows) {
            float v = nan_rows >> q & 1 ? nan_f : o[q] * (1.f / 256.f);
            if (whole) {
              const float sum = c.wsum[0][q] + c.wsum[1][q] + c.wsum[2][q] + c.wsum[3][q];
              p.out.p[c.qout[buf][q] + tid] = __float2bfloat16(sum == 0.f ? 0.f : v / sum);
            } else {
              p.part_o[((long long)g.slot * NT + q) * D + tid] = v;
            }
          }
        }
      }
      if (!whole && warp == 0 && lane < g.nrows)
        p.part_ml[(long long)g.slot * NT + lane] =
            make_float2(run, c.wsum[0][lane] + c.wsum[1][lane] + c.wsum[2][lane] + c.wsum[3][lane]);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.qempty[buf]));
      ++filled;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::kTmemCols);
  }
}

// Joins the partial sums of row tiles that span CTAs: block (c, q) takes row
// q of the row tile that begins in CTA c and ends in a later one, if any.
// The pieces are those of CTAs c, c+1, ... up to the one marked last.
constexpr int kJoinThreads = 256;

template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) kv_attn_join_kernel(const AttnParams p, int grid) {
  constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
  __shared__ int end;
  __shared__ float red[kJoinThreads / 32];
  __shared__ float4 part[kGroups][kLanes];
  __shared__ float part_l[kGroups];
  pdl_launch_dependents();
  pdl_wait();
  const int c0 = blockIdx.x, q = blockIdx.y, tid = threadIdx.x;
  const AttnPiece own = p.pieces[2 * c0 + 1];
  if (!own.valid || q >= own.nrows) return;
  if (tid == 0) end = grid;
  __syncthreads();
  for (int b = c0 + 1; b < grid; b += kJoinThreads) {
    const int k = b + tid;
    if (k < grid && p.pieces[2 * k].valid && p.pieces[2 * k].last) atomicMin(&end, k);
    __syncthreads();
    if (end < grid) break;
    __syncthreads();
  }
  __syncthreads();
  const int n = min(end, grid - 1) - c0 + 1;
  auto slot = [&](int k) { return (long long)(k == 0 ? 2 * c0 + 1 : 2 * (c0 + k)) * NT + q; };
  float m = -3.0e38f;
  for (int k = tid; k < n; k += kJoinThreads) m = fmaxf(m, p.part_ml[slot(k)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red[w]);
  const int gr = tid / kLanes, l = tid % kLanes;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int k = gr; k < n; k += kGroups) {
    const float2 ml = p.part_ml[slot(k)];
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + slot(k) * D + 4 * l);
    const float f = exp2_whole(ml.x - m);
    sum = fmaf(ml.y, f, sum);
    o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
  }
  part[gr][l] = o;
  if (l == 0) part_l[gr] = sum;
  __syncthreads();
  if (tid < kLanes) {
    for (int k = 1; k < kGroups; ++k) {
      const float4 v = part[k][l];
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    sum = 0.f;
    for (int k = 0; k < kGroups; ++k) sum += part_l[k];
    const float f = sum == 0.f ? 0.f : 1.f / sum;
    const int r = own.r0 + q;
    __nv_bfloat16* out = p.out.p + (long long)(own.row0 + r / p.group) * p.out.ts +
                         (long long)(own.h * p.group + r % p.group) * p.out.hs + 4 * l;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
  }
}

}  // namespace sgr
