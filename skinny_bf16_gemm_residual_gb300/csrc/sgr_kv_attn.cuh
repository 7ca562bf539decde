// sgr_kv_attn.cuh -- attention of new tokens over the paged E4M3 cache
// (sgr_attention.h): what its two kernels share -- the work and its split, the
// warp that walks it and loads pages, and the join of partial sums.
//
// The unit of work is a row tile (up to NT query rows that share a key/value
// head: the head's query group, times the new tokens of a sequence) against a
// 128-token tile of the cache.  Every CTA takes the same number of units of
// all sequences and heads, in order, whatever the lengths, and one more unit
// for each row tile, which is what its beginning and end cost (without it CTAs
// with many short sequences finish last: 24.2 against 18.7 us for 32 ragged
// sequences, with weights in two parts).  A row tile that spans CTAs leaves partial sums (o, R, l) in the
// workspace and a second kernel joins them in order (the same bits on every
// run).  For short caches (`whole`) a row tile is one unit and nothing is
// joined.
//
// Both kernels feed the FP8 tensor core (tcgen05.mma kind::f8f6f4) with the
// cache's codes straight from TMA.  The queries are brought into E4M3 as two
// parts, hi = e4m3(b) and lo = e4m3 of the rest, each row scaled by a power of
// two, which holds 8 significant bits; the weights into three (few rows) or
// into FP16 (many).
#pragma once

#include <cuda.h>

#include "sgr_internal.h"
#include "sgr_kv_append.cuh"

namespace sgr {

constexpr int kAttnTile = 128;  // tokens
constexpr int kAttnQueue = 8;   // segments handed out ahead
constexpr int kNap = 64;        // nanoseconds between the polls of roles that mostly wait

// A run of tiles [ta, tb) of one row tile, the unit that the roles work by.
enum : int { kSegStart = 1, kSegEnd = 2, kSegStop = 4 };
struct AttnSeg {
  int kind;
  int h, row0, r0, nrows;  // key/value head; the sequence's first row; rows r0 .. r0+nrows-1 of its n * group
  int first;               // position of the sequence's first row
  int ta, tb;
  int tlo, thi;  // positions that some row of the tile sees
  int slot;      // of its partial sums
  int n, b;      // new tokens of the sequence, its number
};

// Owner of the partial sums of a row tile that begins in a CTA and ends in
// CTA `last` (0: none).
struct AttnPiece {
  int last;
  int h, row0, r0, nrows;
  int pad[3];
};

struct AttnParams {
  KvHeads q, out;
  KvCacheRef cache;
  KvBatch batch;
  float scale_log2;  // scale * log2(e)
  int window;        // INT_MAX: none
  int sinks;         // first positions that stay visible (0 without a window)
  int group;         // query heads a key/value head
  unsigned group_inv;  // floor(2^32 / group), at most 2^32 - 1
  int reuse;         // row tiles of a sequence share the cache's bytes
  int whole;         // a row tile is one unit
  const unsigned long long* tree;  // bits of the new tokens that a row sees, tree_words of them; NULL: those up to its own
  long long tree_stride;
  int tree_words;
  float* lse;  // [rows][query heads], or NULL
  unsigned* err;
  float* part_o;      // [2 grid][NT][D]; row tiles of 256: [2 grid][D / 4][NT][4]
  float2* part_ml;    // [2 grid][NT]  maximum, sum
  AttnPiece* pieces;  // [grid]
};

// Row tile j of a sequence: its rows, the positions they see from the first
// window on (tlo, below it the sinks alone), its tiles, its units (a row tile
// that sees nothing is one unit: its zeros).  Tiles are numbered by position
// from the windows' first on; the sinks' come right before it (TileMap).
struct AttnItem {
  int r0, nrows, tlo, thi, ta, tb, units;
};

// Tile numbers of a row tile -> tiles by position: the tiles between the sinks
// and the windows, `gap` of them, are left out.
struct TileMap {
  int tw, gap;

  // (sinks = 0: the identity)
  __host__ __device__ __forceinline__ TileMap(int tlo, int sinks)
      : tw(tlo / kAttnTile), gap(tw - min((int)(((unsigned)sinks + kAttnTile - 1) / kAttnTile), tw)) {}
  __host__ __device__ __forceinline__ int at(int t) const { return t < tw ? t - gap : t; }
};

// r / group for 0 <= r < 2^31: the product is at most one too small.
__device__ __forceinline__ int div_group(const AttnParams& p, int r) {
  const int q = (int)__umulhi((unsigned)r, p.group_inv);
  return q + (r - q * p.group >= p.group ? 1 : 0);
}

// The last position that the tok-th row of a sequence sees, its own: -1 for any
// padding row, so that last - window (2^31 - 1 for none) stays within 32 bits.
__host__ __device__ __forceinline__ int row_last(int first, int tok) {
  const int pos = first + tok;
  return pos < -1 ? -1 : pos;
}

// Whether a row sees a position, (last - window, last].
__host__ __device__ __forceinline__ bool row_sees(int pos, int last, int window) {
  return pos <= last && pos > last - window;
}

// The first position that a row sees of its row tile's, from tlo on.
__host__ __device__ __forceinline__ int row_first(int tlo, int last, int window) {
  const int lo = last - window + 1;
  return lo < tlo ? tlo : lo;
}

// Whether a row sees a position: in its window, or a sink up to its own.
__host__ __device__ __forceinline__ bool row_sees(int pos, int last, int window, int sinks) {
  return row_sees(pos, last, window) || (pos < sinks && pos <= last);
}

// ------------------------------------------------------------ drafted trees
// A row's bits from the j-th new token on, 32 of them (bits past the last word
// are zeros).
__host__ __device__ __forceinline__ uint32_t tree_bits(const unsigned long long* row, int words, int j) {
  const int w = j >> 6, s = j & 63;
  const unsigned long long lo = w < words ? row[w] : 0ULL, hi = s > 32 && w + 1 < words ? row[w + 1] : 0ULL;
  return (uint32_t)(lo >> s) | (s > 32 ? (uint32_t)(hi << (64 - s)) : 0u);
}

// A row of a tree, the tok-th of n of a sequence: the position that it stands
// for, behind as many as it sees of the new ones but itself (-1: a padding row),
// and whether it sees any of the new ones.
struct TreeRow {
  int last;
  bool drafts;
};

__host__ __device__ __forceinline__ TreeRow tree_row(const AttnParams& p, int row0, int n, int first, int tok) {
  if (first + tok < 0) return {-1, false};
  const unsigned long long* bits = p.tree + (long long)(row0 + tok) * p.tree_stride;
  const int j0 = first < 0 ? -first : 0;  // new tokens before the first position are not there
  int count = 0;
  for (int w = 0; w < p.tree_words && 64 * w < n; ++w) {
    unsigned long long x = bits[w];
    if (n - 64 * w < 64) x &= (1ULL << (n - 64 * w)) - 1;
    if (j0 > 64 * w) x = j0 - 64 * w < 64 ? x >> (j0 - 64 * w) << (j0 - 64 * w) : 0ULL;
#ifdef __CUDA_ARCH__
    count += __popcll(x);
#else
    count += __builtin_popcountll(x);
#endif
  }
  return {max(first, 0) + max(count - 1, 0), count > 0};
}

// Bits of the positions x .. x + 31 that lie in [lo, hi].
__host__ __device__ __forceinline__ uint32_t span_bits(int x, int lo, int hi) {
  const int a = max(lo - x, 0), b = min(hi - x, 31);
  return a > b ? 0u : (0xffffffffu >> (31 - b)) & (0xffffffffu << a);
}

// Bits of the positions x .. x + 31 (x >= 0) that a row with this `last` sees;
// thi: behind the sequence's last position, first: its first new one.
__host__ __device__ __forceinline__ uint32_t row_bits(const AttnParams& p, int x, int last, int thi, int first, int row) {
  uint32_t m = span_bits(x, max(last - p.window + 1, 0), last) | span_bits(x, 0, min(last, p.sinks - 1));
  if (p.tree && x + 31 >= first) {
    m &= span_bits(x, 0, first - 1);
    if (last >= 0) {
      const unsigned long long* bits = p.tree + (long long)row * p.tree_stride;
      const int j = x - first;
      const uint32_t t = j >= 0 ? tree_bits(bits, p.tree_words, j) : tree_bits(bits, p.tree_words, 0) << -j;
      m |= t & span_bits(x, 0, thi - 1);
    }
  }
  return m;
}

template <int NT, bool kMasked>
__device__ __forceinline__ AttnItem attn_item(const AttnParams& p, const KvSeq& s, int j) {
  AttnItem it;
  it.r0 = j * NT;
  it.nrows = min(NT, s.n * p.group - it.r0);
  // (every row of a tree may see all of its new tokens, and stands for the first one's position at least)
  const int first = s.len - s.n, p0 = kMasked && p.tree ? first : first + div_group(p, it.r0);
  it.thi = max(kMasked && p.tree ? s.len : first + div_group(p, max(it.r0 + it.nrows - 1, 0)) + 1, 0);
  it.tlo = p.window > p0 ? 0 : p0 - p.window + 1;
  it.ta = it.thi <= 0 ? 0 : kMasked ? TileMap(it.tlo, p.sinks).gap : it.tlo / kAttnTile;
  it.tb = (it.thi + kAttnTile - 1) / kAttnTile;
  it.units = p.whole || it.tb <= it.ta ? 1 : it.tb - it.ta + 1;  // the first for its beginning and end
  return it;
}

template <int NT, bool kMasked>
__device__ __forceinline__ int attn_seq_units(const AttnParams& p, const KvSeq& s) {
  int u = 0;
  for (int j = 0; j * NT < s.n * p.group; ++j) u += attn_item<NT, kMasked>(p, s, j).units;
  return u;
}

// The warp that walks a CTA's share of the work: finds it, hands out its
// segments, loads the pages of its tiles by TMA (V, then K, of a stage of the
// ring; without Ctl::kValues K alone) and writes their scales beside them.  Rows
// that see nothing get their zeros here.  Executed by one whole warp.
template <int D, int NT, bool kMasked, class Ctl>
__device__ __forceinline__ void attn_walk(Ctl& c, const AttnParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                          uint32_t ring) {
  constexpr bool kValues = Ctl::kValues;
  constexpr int S = Ctl::kStages, M = Ctl::kMeta, kTile = kAttnTile * D, kStage = (kValues ? 2 : 1) * kTile;
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &c.abort;
  // ------------------------------------------------ this CTA's share of the work
  // CTA c of `active` takes the units [begin(c), begin(c + 1)) of all
  // sequences: the first `rest` CTAs one more than `per`.  (The host refuses
  // what might not fit 31 bits.)
  const int ps = p.cache.page_shift, hk = p.cache.heads;
  int b = 0, h = 0, j = 0, skip = 0, u = 0, u1 = 0, per = 0, rest = 0;
  KvSeq s{0, 0, 0};
  {
    // Each lane counts its (consecutive) sequences; or, where few sequences have
    // many row tiles, the lanes count a sequence's together, one sequence after
    // another (two chunks of 16 row tiles a head: 3 us less to the first tile).
    const int per_lane = (p.batch.batch + 31) / 32, b_first = lane * per_lane;
    const int b_last = min(b_first + per_lane, p.batch.batch);
    int mine = 0, units = 0;
    int tiles = 0;  // row tiles of a sequence, the most of any
    // (Tiles of fewer rows are one a sequence, or a few where the work does not fill
    // the GPU: the plan takes them while row tiles times tiles are at most two for
    // each SM.)
    constexpr bool kSeveral = NT >= 32;
    if (kSeveral && p.reuse && per_lane == 1) {
      if (b_first < b_last) s = kv_seq(p.batch, ps, b_first, p.err);
      tiles = __reduce_max_sync(0xffffffffu, (s.n * p.group + NT - 1) / NT);
    }
    if (kSeveral && tiles > 2 * p.batch.batch * ((tiles + 31) / 32)) {
      for (int x = 0; x < p.batch.batch; ++x) {
        const KvSeq sx{__shfl_sync(0xffffffffu, s.row0, x), __shfl_sync(0xffffffffu, s.n, x), __shfl_sync(0xffffffffu, s.len, x)};
        int part = 0;
        for (int k = lane; k * NT < sx.n * p.group; k += 32) part += attn_item<NT, kMasked>(p, sx, k).units;
        part = __reduce_add_sync(0xffffffffu, part);
        if (lane == x) {
          units = part;
          mine = units * hk;
        }
      }
    } else {
#pragma unroll 4
      for (int x = b_first; x < b_last; ++x) {
        s = kv_seq(p.batch, ps, x, p.err);
        units = attn_seq_units<NT, kMasked>(p, s);
        mine += units * hk;
      }
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31);
    // (with fewer units than CTAs the last ones have none, the others one each)
    const int active = min(total, (int)gridDim.x), c0 = (int)blockIdx.x;
    if (c0 < active) {
      per = total / active;
      rest = total - per * active;
      u = c0 * per + min(c0, rest);
      u1 = u + per + (c0 < rest ? 1 : 0);
      const int before = upto - mine;
      const int src = __ffs(__ballot_sync(0xffffffffu, u >= before && u < upto)) - 1;
      int off = u - __shfl_sync(0xffffffffu, before, max(src, 0));
      // (row offsets that run backwards may count more units than 31 bits hold)
      bool found = src >= 0;
      b = max(src, 0) * per_lane;
      if (per_lane == 1) {  // the lane still has its only sequence
        s.row0 = __shfl_sync(0xffffffffu, s.row0, b);
        s.n = __shfl_sync(0xffffffffu, s.n, b);
        s.len = __shfl_sync(0xffffffffu, s.len, b);
        units = __shfl_sync(0xffffffffu, units, b);
      } else {
        for (; found; ++b) {
          if (b >= p.batch.batch) found = false;
          if (!found) break;
          s = kv_seq(p.batch, ps, b, nullptr);
          units = attn_seq_units<NT, kMasked>(p, s);
          if (off < units * hk) break;
          off -= units * hk;
        }
      }
      if (!found) u1 = u, off = 0, units = 1;
      h = off / units;
      off -= h * units;
      // The row tile: the lanes look at 32 of them at once.
      if (kSeveral && p.reuse) {
        while (found && j * NT < s.n * p.group) {
          const int each = (j + lane) * NT < s.n * p.group ? attn_item<NT, kMasked>(p, s, j + lane).units : 0;
          int upto_j = each;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, upto_j, o);
            if (lane >= o) upto_j += up;
          }
          const unsigned past = __ballot_sync(0xffffffffu, upto_j > off);
          if (past) {
            const int at = __ffs(past) - 1;
            off -= __shfl_sync(0xffffffffu, upto_j - each, at);
            j += at;
            break;
          }
          off -= __shfl_sync(0xffffffffu, upto_j, 31);
          j += 32;
        }
      } else {
        for (int x; found && off >= (x = attn_item<NT, kMasked>(p, s, j).units); ++j) off -= x;
      }
      skip = off;
    }
  }
  auto cta_of = [&](int x) {  // the CTA that takes unit x
    const int y = rest * (per + 1);
    return x < y ? x / (per + 1) : rest + (x - y) / per;
  };
  // ------------------------------------------------------- walk and TMA loads
  const uint64_t policy = p.reuse ? policy_evict_last() : policy_evict_first();
  int sq = 0;
  AttnItem it{};
  bool ok = true;
  AttnPiece piece{};  // of the row tile that goes on in the next CTA
  if (u < u1) it = attn_item<NT, kMasked>(p, s, j);
  int t = 0, t_end = 0;  // tiles of the segment handed out last
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_wait_nap<kNap>(smem_u32(bar), parity, abort_flag)) {
      if (!*abort_flag) report_error(p.err, kErrWaitEmpty);
      *abort_flag = 1;
      ok = false;
    }
    ok = __all_sync(0xffffffffu, ok);
  };
  auto hand_out = [&](const AttnSeg& g) {
    const int qi = sq % kAttnQueue;
    wait(&c.segempty[qi], ((sq / kAttnQueue) & 1) ^ 1);
    if (!ok) return;
    if (lane == 0) {
      c.seg[qi] = g;
      mbar_arrive(smem_u32(&c.segfull[qi]));
    }
    ++sq;
  };
  struct Tile {
    int h, flags;
    int live0, live1;  // its tokens that some row sees
    int page;          // this lane's table entry, -1 = none
    int src;           // the lane that has its scales (kBatch)
    float ks, vs;
  };
  // For row tiles of many rows pages and scales come for all the tiles at once
  // that 32 lanes have pages of (lane = one page), and those of the next batch
  // while this one is used.  For few rows they come a tile ahead, across the ends
  // of sequences, of which there is one every few tiles there (32 sequences of up
  // to 4096: 19.8 us so, 20.8 in batches).
  constexpr bool kBatch = NT >= 128;
  struct Pages {
    int page;
    float ks, vs;
  };
  const int per_tile = kAttnTile >> ps, batch = 32 / per_tile;  // pages a tile, tiles a batch
  Pages here{}, ahead{};
  int first_tile = 0;
  bool fresh = true;  // whether no batch of the segment has been asked for
  AttnItem cur{};
  int cur_h = 0, cur_b = 0, cur_p0 = 0, cur_p1 = 0;
  // This lane's page of the batch from tile t0 on, -1 where there is none.
  auto ask_pages = [&](int t0, Pages& g) {
    const bool there = t0 + lane / per_tile < t_end;
    const int tile = there ? t0 + lane / per_tile : t_end - 1;
    const int x0 = (kMasked ? TileMap(cur.tlo, p.sinks).at(tile) : tile) * kAttnTile;
    const int block = (x0 >> ps) + lane % per_tile, at = block << ps;
    if (there && at < cur.thi && (at + (1 << ps) > cur.tlo || (kMasked && at < p.sinks)))
      g.page = p.batch.table[(long long)cur_b * p.batch.table_stride + block];
    else
      g.page = -2;  // (not asked for)
  };
  auto ask_scales = [&](Pages& g) {
    if (g.page != -2 && (g.page < 0 || g.page >= p.cache.num_pages)) {
      report_error(p.err, kErrIndex);
      g.page = -1;
    }
    g.ks = g.vs = 1.f;
    if (g.page >= 0) {
      const long long at = (long long)g.page * p.cache.scale_stride + cur_h;
      g.ks = p.cache.k_scale[at];
      if (kValues) g.vs = p.cache.v_scale[at];
    }
  };
  // The next tile of this CTA's share; hands out the segments it enters.
  auto next_tile = [&](Tile& x) -> bool {
    while (t == t_end) {
      if (u >= u1 || !ok) return false;
      if (it.nrows <= 0) {  // past the last row tile of the head
        j = 0;
        if (s.n == 0 || ++h == hk) {
          h = 0;
          do {
            if (++b >= p.batch.batch) return false;
            s = kv_seq(p.batch, ps, b, nullptr);
          } while (s.n == 0);
        }
        it = attn_item<NT, kMasked>(p, s, 0);
      }
      const int units = it.units, take = min(u1 - u, units - skip);
      u += take;
      if (it.tb <= it.ta) {  // rows that see nothing: zeros
        for (int e = lane; kValues && e < it.nrows * (D / 8); e += 32) {
          const int r = it.r0 + e / (D / 8), tok = div_group(p, r);
          *reinterpret_cast<uint4*>(p.out.p + (long long)(s.row0 + tok) * p.out.ts +
                                    (long long)(h * p.group + r - tok * p.group) * p.out.hs + e % (D / 8) * 8) =
              make_uint4(0u, 0u, 0u, 0u);
          if (kMasked && p.lse && e % (D / 8) == 0)
            p.lse[(long long)(s.row0 + tok) * p.q.heads + h * p.group + r - tok * p.group] = -INFINITY;
        }
        it = attn_item<NT, kMasked>(p, s, ++j);
        continue;
      }
      AttnSeg g;
      g.ta = p.whole ? it.ta : it.ta + max(skip - 1, 0);
      g.tb = p.whole ? it.tb : it.ta + skip + take - 1;
      if (g.tb <= g.ta) continue;  // the share ends with the first unit: no tile
      g.kind = (g.ta == it.ta ? kSegStart : 0) | (skip + take == units ? kSegEnd : 0);
      g.h = h;
      g.row0 = s.row0;
      g.r0 = it.r0;
      g.nrows = it.nrows;
      g.first = s.len - s.n;
      g.tlo = it.tlo;
      g.thi = it.thi;
      g.slot = 2 * (int)blockIdx.x + (g.kind & kSegStart ? 1 : 0);
      g.n = s.n;
      g.b = b;
      hand_out(g);
      if (!ok) return false;
      if (kValues && g.kind == kSegStart) piece = {cta_of(u + units - skip - take - 1), h, s.row0, it.r0, it.nrows, {0, 0, 0}};
      t = g.ta;
      t_end = g.tb;
      fresh = true;
      cur = it;
      cur_h = h;
      cur_b = b;
      cur_p0 = kMasked && p.tree ? g.first - 1 : g.first + div_group(p, it.r0);  // rows see the same up to it, but for windows
      cur_p1 = it.thi - 1;
      skip = 0;
      if (g.kind & kSegEnd) it = attn_item<NT, kMasked>(p, s, ++j);
    }
    const TileMap tm(cur.tlo, kMasked ? p.sinks : 0);
    const bool sink = kMasked && t < tm.tw;  // a tile before the windows: rows see its sinks alone
    const int x0 = (kMasked ? tm.at(t) : t) * kAttnTile, x1 = x0 + kAttnTile;
    ++t;
    x.h = cur_h;
    if (sink) {
      x.live0 = 0;
      x.live1 = min(p.sinks - x0, kAttnTile);
      x.flags = x.live1 < kAttnTile ? 1 : 0;
    } else {
      x.live0 = max(cur.tlo - x0, 0);
      x.live1 = min(cur.thi - x0, kAttnTile);
      x.flags = (x0 < cur.tlo || x1 > cur.thi) ? 1 : 0;
      if (min(x1, cur.thi) - 1 > max(cur_p0, -1) || max(x0, cur.tlo) < (long long)cur_p1 - p.window + 1) x.flags |= 2;
      if (kMasked && x.live0 > 0 && p.sinks > x0) {  // sinks and windows in one tile, perhaps with a gap
        x.live0 = 0;
        x.flags |= 2;
      }
    }
    // Its pages, where some row sees a position of them.
    if constexpr (!kBatch) {
      const int block = (x0 >> ps) + lane, at = block << ps;
      x.page = -2;
      if (lane < per_tile && at < cur.thi && (at + (1 << ps) > cur.tlo || (kMasked && at < p.sinks)))
        x.page = p.batch.table[(long long)cur_b * p.batch.table_stride + block];
      return true;
    }
    int k = t - 1 - first_tile;
    if (fresh) {
      first_tile = t - 1;
      k = 0;
      ask_pages(first_tile, here);
      ask_scales(here);
      fresh = false;
    } else if (k == batch) {
      here = ahead;
      first_tile += batch;
      k = 0;
    }
    if (k == 0) ask_pages(first_tile + batch, ahead);
    if (k == 2) ask_scales(ahead);
    x.src = (k * per_tile + lane) & 31;
    x.page = __shfl_sync(0xffffffffu, here.page, x.src);
    if (lane >= per_tile) x.page = -1;
    return true;
  };
  // Checks this lane's page and asks for its scales (few rows).
  auto load_scales = [&](Tile& x) {
    if (x.page != -2 && (x.page < 0 || x.page >= p.cache.num_pages)) {
      report_error(p.err, kErrIndex);
      x.page = -1;
    }
    x.ks = x.vs = 1.f;
    if (x.page >= 0) {
      const long long at = (long long)x.page * p.cache.scale_stride + x.h;
      x.ks = p.cache.k_scale[at];
      if (kValues) x.vs = p.cache.v_scale[at];
    }
  };
  // One tile ahead of the copies: its table entries are asked for before this
  // tile's scales arrive, which reach the stage behind its copies.
  Tile a{}, next{};
  bool has = next_tile(a);
  if (!kBatch && has) load_scales(a);
  int i = 0, slot = 0;
  uint32_t par = 0;
  const uint32_t page_bytes = (uint32_t)D << ps;
  while (has && ok) {
    if (i >= S) wait(&c.empty[slot], par ^ 1u);
    if (!ok) break;
    const unsigned live = __ballot_sync(0xffffffffu, a.page >= 0);
    const uint32_t kb = smem_u32(&c.kfull[slot]);
    if (lane == 0) {
      mbar_expect_tx(kb, (uint32_t)__popc(live) * page_bytes);
      if constexpr (kValues) mbar_arrive_expect_tx(smem_u32(&c.vfull[slot]), (uint32_t)__popc(live) * page_bytes);
    }
    __syncwarp();
    if (a.page >= 0) {
      const uint32_t dst = ring + (uint32_t)slot * kStage + (uint32_t)lane * page_bytes;
      tma_load_4d(dst + kStage - kTile, &tmK, 0, 0, a.h, a.page, kb, policy);
      if constexpr (kValues) tma_load_4d(dst, &tmV, 0, 0, a.h, a.page, smem_u32(&c.vfull[slot]), policy);
    }
    const int meta = i % M;
    if constexpr (kBatch) {
      a.ks = __shfl_sync(0xffffffffu, here.ks, a.src);
      a.vs = __shfl_sync(0xffffffffu, here.vs, a.src);
    } else {
      has = next_tile(next);
    }
    if (lane < per_tile) {
      c.kscale[meta][lane] = a.ks;
      // (an exponent of -inf marks a page that is not there)
      if constexpr (kValues)
        c.vexp[meta][lane] = a.page >= 0 ? (float)((int)((__float_as_uint(a.vs) >> 23) & 0xFF) - 127) : -INFINITY;
      else
        c.page[meta][lane] = a.page;
    }
    if (lane == 0) {
      c.flags[meta] = (a.flags & 3) | (__popc(live) < per_tile ? 1 : 0);
      c.live[meta][0] = a.live0;
      c.live[meta][1] = a.live1;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(kb);
    ++i;
    if (++slot == S) {
      slot = 0;
      par ^= 1u;
    }
    if constexpr (kBatch) {
      has = next_tile(a);
    } else {
      a = next;
      if (has) load_scales(a);
    }
  }
  bool stopped = false;
  if constexpr (Ctl::kStopStage) if (ok) {  // a stage that ends the sequence
    if (i >= S) wait(&c.empty[slot], par ^ 1u);
    stopped = ok;
    if (ok && lane == 0) {
      c.flags[i % M] = 8;
      mbar_arrive(smem_u32(&c.kfull[slot]));
      mbar_arrive(smem_u32(&c.vfull[slot]));
    }
  }
  AttnSeg stop{};
  stop.kind = kSegStop;
  hand_out(stop);
  if (kValues && lane == 0) p.pieces[blockIdx.x] = piece;
  // Every copy that this warp issued lands before the CTA may exit.  (The
  // stage that the stop took was empty: its copies have landed.)
  bool landed = true;
  for (int k = max(i - S + (stopped ? 1 : 0), 0); k < i && landed; ++k) {
    landed = mbar_wait(smem_u32(&c.kfull[k % S]), (k / S) & 1);
    if constexpr (kValues) landed = landed && mbar_wait(smem_u32(&c.vfull[k % S]), (k / S) & 1);
  }
  if (!landed) report_error(p.err, kErrDrain);
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

// Pairs of FP32 values, one instruction for both.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_parts(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Eight elements (of a BF16 row held by kLanes neighbouring lanes) as hi and lo
// codes, b = hi + lo / lo_scale, b = x * sign / factor with the row's largest
// |b| in [128, 256).  A row with an infinity or NaN gets a NaN factor.
struct QuerySplit {
  uint2 hi, lo;
  float factor;
};

// Two values as hi and lo codes, a pair of bytes each.
__device__ __forceinline__ void split_pair(float a, float b, float lo_scale, uint32_t& hi, uint32_t& lo) {
  asm("{\n\t.reg .b16 h, l, z;\n\t.reg .b32 x, y, f;\n\t"
      "cvt.rn.f16x2.f32 x, %3, %2;\n\t"
      "cvt.rn.f16x2.f32 f, %4, %4;\n\t"
      "mov.b16 z, 0;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 h, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, h;\n\t"
      "sub.rn.f16x2 x, x, y;\n\t"
      "mul.rn.f16x2 x, x, f;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 l, x;\n\t"
      "mov.b32 %0, {h, z};\n\t"
      "mov.b32 %1, {l, z};\n\t}"
      : "=r"(hi), "=r"(lo)
      : "f"(a), "f"(b), "f"(lo_scale));
}

template <int kLanes>
__device__ __forceinline__ QuerySplit split_query(const uint4& v, float sign, float lo_scale) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t mag = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) mag = max(mag, max(u[k] & 0x7FFFu, (u[k] >> 16) & 0x7FFFu));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, o));
  const int ex = (int)(mag >> 7);  // biased exponent of the row's largest magnitude
  int k = ex == 0 ? 126 : 134 - ex;
  k = min(max(k, -120), 126);
  const float sc = kv_exp2i(k) * sign;
  float x[8];
  unpack8(v, x);
  // In FP16 on the way: its 11 bits hold b (8 bits) down to 2^-17, far below what
  // E4M3 rounds to zero, and the rest times lo_scale exactly.
  uint32_t part[2][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) split_pair(x[2 * e] * sc, x[2 * e + 1] * sc, lo_scale, part[0][e], part[1][e]);
  QuerySplit s;
  s.hi = make_uint2(part[0][0] | part[0][1] << 16, part[0][2] | part[0][3] << 16);
  s.lo = make_uint2(part[1][0] | part[1][1] << 16, part[1][2] | part[1][3] << 16);
  s.factor = ex == 255 ? __int_as_float(0x7fffffff) : kv_exp2i(-k);
  return s;
}

// Whether any thread of a named barrier's says so.
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t threads, bool x) {
  uint32_t any;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)x), "r"(id), "r"(threads)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ void sts8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Logarithm of the sum of a row's exponentials, from its R and the sum of its
// weights (256 p: the 8).  The sum has 24 bits and R is whole, so it is good to
// some 2^-23 of the larger of itself and 1.
__device__ __forceinline__ float log_sum_exp(float R, float sum) {
  return sum == 0.f ? -INFINITY : (R - 8.f + log2f(sum)) * 0.6931471805599453f;
}

// Joins the partial sums of row tiles that span CTAs: blocks x = c take the row
// tile that begins in CTA c and ends in a later one, if any; its pieces are
// those of CTAs c, c + 1, ..., last.  A row is joined by kParts warps, each
// taking every kParts-th run of pieces with all its reads under way at once
// (one memory round trip for the owner, one for the pieces: few long sequences
// have tens of pieces a row), in a fixed order.
//
//     o = sum_k 2^(R_k - m) o_k / sum_k 2^(R_k - m) l_k,   m = max_k R_k
//
// Bound: the latency of its launch and of those two round trips, some 3 us of
// a call.
constexpr int kJoinThreads = 256;

template <int NT>
struct JoinShape {
  static constexpr int kParts = NT <= 16 ? 4 : 1;  // warps a row
  static constexpr int kRows = kJoinThreads / 32 / kParts;
  static constexpr int kRun = 8;  // pieces read at once
};

template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) kv_attn_join_kernel(const AttnParams p) {
  constexpr int kE = D / 32, kParts = JoinShape<NT>::kParts, kRows = JoinShape<NT>::kRows;  // kE: elements a lane
  constexpr int kRun = JoinShape<NT>::kRun;
  __shared__ float part_o[kRows][kParts][D];
  __shared__ float2 part_ml[kRows][kParts];
  pdl_launch_dependents();
  pdl_wait();
  const int c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = warp / kParts, part = warp % kParts, q = blockIdx.y * kRows + row;
  const AttnPiece own = p.pieces[c0];
  if (own.last <= c0 || q >= own.nrows) return;  // (all warps of the row)
  const int n = own.last - c0 + 1;
  auto slot = [&](int k) { return (long long)(k == 0 ? 2 * c0 + 1 : 2 * (c0 + k)) * NT + q; };
  float m = -3.0e38f, sum = 0.f, o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = 0.f;
  for (int k0 = kRun * part; k0 < n; k0 += kRun * kParts) {
    float v[kRun][kE];
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const float* at = p.part_o + slot(min(k0 + k, n - 1)) * D + lane * kE;
      if constexpr (kE == 4) {
        const float4 u = *reinterpret_cast<const float4*>(at);
        v[k][0] = u.x, v[k][1] = u.y, v[k][2] = u.z, v[k][3] = u.w;
      } else {
        const float2 u = *reinterpret_cast<const float2*>(at);
        v[k][0] = u.x, v[k][1] = u.y;
      }
    }
    float2 ml = make_float2(-3.0e38f, 0.f);  // lane k: of piece k0 + k
    if (lane < kRun && k0 + lane < n) ml = p.part_ml[slot(k0 + lane)];
    const float now = fmaxf(m, warp_max(ml.x)), old = exp2_whole(m - now);
    const float f = lane < kRun && k0 + lane < n ? exp2_whole(ml.x - now) : 0.f;
    m = now;
    sum *= old;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] *= old;
    const float w = ml.y * f;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      if (k0 + k >= n) break;
      const float fk = __shfl_sync(0xffffffffu, f, k);
      sum += __shfl_sync(0xffffffffu, w, k);
#pragma unroll
      for (int e = 0; e < kE; ++e) o[e] = fmaf(v[k][e], fk, o[e]);
    }
  }
  if constexpr (kParts > 1) {
#pragma unroll
    for (int e = 0; e < kE; ++e) part_o[row][part][lane * kE + e] = o[e];
    if (lane == 0) part_ml[row][part] = make_float2(m, sum);
    __syncwarp();
    named_bar_sync(1 + row, 32 * kParts);
    if (part > 0) return;
    float all = m;
#pragma unroll
    for (int k = 1; k < kParts; ++k) all = fmaxf(all, part_ml[row][k].x);
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = 0.f;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      if (kRun * k >= n) break;  // (a part without pieces)
      const float f = exp2_whole(part_ml[row][k].x - all);
      sum = fmaf(part_ml[row][k].y, f, sum);
#pragma unroll
      for (int e = 0; e < kE; ++e) o[e] = fmaf(part_o[row][k][lane * kE + e], f, o[e]);
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  const int r = own.r0 + q, tok = div_group(p, r);
  if (p.lse && lane == 0) {
    if constexpr (kParts > 1) {
      m = part_ml[row][0].x;
#pragma unroll
      for (int k = 1; k < kParts; ++k) m = fmaxf(m, part_ml[row][k].x);
    }
    p.lse[(long long)(own.row0 + tok) * p.q.heads + own.h * p.group + r - tok * p.group] = log_sum_exp(m, sum);
  }
  __nv_bfloat16* out = p.out.p + (long long)(own.row0 + tok) * p.out.ts +
                       (long long)(own.h * p.group + r - tok * p.group) * p.out.hs + lane * kE;
  if constexpr (kE == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f));
  else
    *reinterpret_cast<uint32_t*>(out) = pack_bf16(o[0] * f, o[1] * f);
}

}  // namespace sgr
