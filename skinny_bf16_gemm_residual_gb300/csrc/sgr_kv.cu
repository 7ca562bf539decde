// sgr_kv.cu -- C ABI of the attention operators (include/sgr_attention.h):
// argument checks, device set-up and kernel launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>

#include "sgr_attention.h"
#include "sgr_internal.h"
#include "sgr_kv_append.cuh"
#include "sgr_kv_attn_few.cuh"
#include "sgr_kv_attn_rows.cuh"

namespace {

using sgr::kMaxDevices;

constexpr long long kMaxStride = 1LL << 36;  // as the row strides of skinny_gemm_residual.h
constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxHeads = 1 << 12;
constexpr int kMaxGroup = 1 << 10;  // query heads a key/value head: rows of a sequence stay below 2^30

// ------------------------------------------------------------ argument checks
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Extent {
  uintptr_t lo, hi;  // [lo, hi) bytes
};

bool overlap(Extent a, Extent b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

Extent heads_extent(const sgr_heads& x, long long tokens, int dim) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(x.data);
  if (tokens <= 0 || x.heads <= 0) return {b, b};
  return {b, b + 2 * static_cast<uintptr_t>((tokens - 1) * x.token_stride + (x.heads - 1) * x.head_stride + dim)};
}

// Whether two sets of head rows share elements.  Slices of one packed buffer
// (same token stride, each row's heads within it) are told apart by their
// place in the row; anything else by its extent.
bool heads_overlap(const sgr_heads& a, const sgr_heads& b, long long tokens, int dim) {
  if (!overlap(heads_extent(a, tokens, dim), heads_extent(b, tokens, dim))) return false;
  const long long ts = a.token_stride;
  const long long wa = (a.heads - 1) * a.head_stride + dim, wb = (b.heads - 1) * b.head_stride + dim;
  if (ts != b.token_stride || wa > ts || wb > ts) return true;
  const long long bytes = (long long)(reinterpret_cast<intptr_t>(b.data) - reinterpret_cast<intptr_t>(a.data));
  const long long d = ((bytes % (2 * ts) + 2 * ts) % (2 * ts)) / 2;  // place of b's heads in a's rows
  return d < wa || d + wb > ts;
}

bool same_rows(const sgr_heads& a, const sgr_heads& b) {
  return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride && a.heads == b.heads;
}

int check_heads(const sgr_heads* x, int heads, int dim, bool output) {
  if (!x) return SGR_ERR_NULL;
  if (x->reserved != 0) return SGR_ERR_UNSUPPORTED;
  if (x->heads < 1 || x->heads != heads) return SGR_ERR_SHAPE;
  if (heads > kMaxHeads) return SGR_ERR_UNSUPPORTED;
  if (!x->data) return SGR_ERR_NULL;
  if (x->token_stride < 0 || x->head_stride < 0) return SGR_ERR_SHAPE;
  if (x->token_stride > kMaxStride || x->head_stride > kMaxStride) return SGR_ERR_UNSUPPORTED;
  if (!aligned(x->data, 16) || x->token_stride % 8 || x->head_stride % 8) return SGR_ERR_ALIGN;
  // Rows that are written must not overlap one another: heads within a token
  // or tokens within a head.
  const long long ts = x->token_stride, hs = x->head_stride;
  if (hs < dim && heads > 1) return SGR_ERR_SHAPE;
  if (output && ts < dim) return SGR_ERR_SHAPE;
  return SGR_OK;
}

// Outputs: neither tokens within heads nor heads within tokens may collide.
int check_rows(const sgr_heads& x, long long tokens, int dim) {
  if (tokens <= 1) return SGR_OK;
  const long long ts = x.token_stride, hs = x.head_stride;
  if (x.heads == 1) return ts >= dim ? SGR_OK : SGR_ERR_SHAPE;
  const bool heads_inside = ts >= (x.heads - 1) * hs + dim, tokens_inside = hs >= (tokens - 1) * ts + dim;
  return heads_inside || tokens_inside ? SGR_OK : SGR_ERR_SHAPE;
}

int check_norm_rope(const sgr_norm_rope* nr, int dim) {
  if (!nr) return SGR_ERR_NULL;
  if ((nr->q_weight && !aligned(nr->q_weight, 16)) || (nr->k_weight && !aligned(nr->k_weight, 16)))
    return SGR_ERR_ALIGN;
  if ((nr->q_weight || nr->k_weight) && !(nr->eps >= 0.f && std::isfinite(nr->eps))) return SGR_ERR_SHAPE;
  if (nr->table) {
    if (!aligned(nr->table, 16)) return SGR_ERR_ALIGN;
    if (nr->table_rows < 1 || nr->rot_dim < 16 || nr->rot_dim % 16 || nr->rot_dim > dim) return SGR_ERR_SHAPE;
  }
  return SGR_OK;
}

int check_dim(int dim) {
  if (dim < 1) return SGR_ERR_SHAPE;
  return dim == 64 || dim == 128 ? SGR_OK : SGR_ERR_UNSUPPORTED;
}

int validate_rope(const sgr_heads* q, const sgr_heads* k, const sgr_heads* qo, const sgr_heads* ko,
                  const int* positions, int tokens, int dim, const sgr_norm_rope* nr) {
  int rc;
  if (tokens < 0) return SGR_ERR_SHAPE;
  if ((rc = check_dim(dim)) != SGR_OK) return rc;
  if (tokens > kMaxTokens) return SGR_ERR_UNSUPPORTED;
  if (!q || !qo || (k == nullptr) != (ko == nullptr)) return SGR_ERR_NULL;
  if (tokens == 0) return SGR_OK;
  if (!positions) return SGR_ERR_NULL;
  if (!aligned(positions, 4)) return SGR_ERR_ALIGN;
  if ((rc = check_norm_rope(nr, dim)) != SGR_OK) return rc;
  const sgr_heads* in[2] = {q, k};
  const sgr_heads* out[2] = {qo, ko};
  for (int i = 0; i < (k ? 2 : 1); ++i) {
    if ((rc = check_heads(in[i], in[i]->heads, dim, false)) != SGR_OK) return rc;
    if ((rc = check_heads(out[i], in[i]->heads, dim, true)) != SGR_OK) return rc;
    if ((rc = check_rows(*out[i], tokens, dim)) != SGR_OK) return rc;
  }
  for (int i = 0; i < (k ? 2 : 1); ++i)
    for (int j = 0; j < (k ? 2 : 1); ++j) {
      if (!(i == j && same_rows(*in[i], *out[j])) && heads_overlap(*in[i], *out[j], tokens, dim)) return SGR_ERR_ALIAS;
      if (i < j && heads_overlap(*out[i], *out[j], tokens, dim)) return SGR_ERR_ALIAS;
    }
  return SGR_OK;
}

int check_cache(const sgr_kv_cache* c) {
  if (!c) return SGR_ERR_NULL;
  int rc;
  if ((rc = check_dim(c->head_dim)) != SGR_OK) return rc;
  if (c->num_pages < 0 || c->heads < 1 || c->page_size < 1) return SGR_ERR_SHAPE;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return SGR_ERR_UNSUPPORTED;
  if (c->heads > kMaxHeads) return SGR_ERR_UNSUPPORTED;
  if (c->num_pages == 0) return SGR_OK;  // a cache without pages: block tables name none
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return SGR_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return SGR_ERR_ALIGN;
  struct Dim {
    long long stride, count;
  } d[3] = {{c->token_stride, c->page_size}, {c->head_stride, c->heads}, {c->page_stride, c->num_pages}};
  for (const Dim& x : d) {
    if (x.count > 1 && x.stride < 0) return SGR_ERR_SHAPE;
    if (x.stride > kMaxStride) return SGR_ERR_UNSUPPORTED;
    if (x.count > 1 && x.stride % 16) return SGR_ERR_ALIGN;
  }
  // Positions must not overlap: from the smallest stride up, each at least
  // the span of what lies inside it.
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (d[j].stride > d[j + 1].stride) std::swap(d[j], d[j + 1]);
  long long span = c->head_dim;
  for (const Dim& x : d)
    if (x.count > 1) {
      if (x.stride < span) return SGR_ERR_SHAPE;
      span += (x.count - 1) * x.stride;
    }
  if (c->scale_stride < c->heads && c->num_pages > 1) return SGR_ERR_SHAPE;
  if (c->scale_stride > kMaxStride) return SGR_ERR_UNSUPPORTED;
  return SGR_OK;
}

long long cache_bytes(const sgr_kv_cache& c) {
  return (c.num_pages - 1) * c.page_stride + (c.heads - 1) * c.head_stride + (c.page_size - 1) * c.token_stride +
         c.head_dim;
}

int check_batch(const sgr_kv_batch* b) {
  if (!b) return SGR_ERR_NULL;
  if (b->batch < 0 || b->tokens < 0 || b->max_new < 0 || b->max_pages < 0) return SGR_ERR_SHAPE;
  if (b->batch > kMaxTokens || b->tokens > kMaxTokens || b->max_pages > (1 << 24)) return SGR_ERR_UNSUPPORTED;
  if (b->batch == 0 || b->tokens == 0) return SGR_OK;
  if (!b->q_start && b->tokens != b->batch) return SGR_ERR_SHAPE;
  if (b->max_new < 1 || b->table_stride < b->max_pages) return SGR_ERR_SHAPE;
  if (!b->seq_len || (b->max_pages > 0 && !b->block_table)) return SGR_ERR_NULL;
  if (!aligned(b->seq_len, 4) || !aligned(b->block_table, 4) || !aligned(b->q_start, 4)) return SGR_ERR_ALIGN;
  if (b->table_stride > kMaxStride) return SGR_ERR_UNSUPPORTED;
  return SGR_OK;
}

bool empty(const sgr_kv_batch& b) { return b.batch == 0 || b.tokens == 0; }

// Whether rows of heads and the cache (codes or scales) share memory.
bool touches_cache(const sgr_heads& x, const sgr_kv_cache& c, long long tokens) {
  if (c.num_pages == 0) return false;
  const Extent e = heads_extent(x, tokens, c.head_dim);
  for (const void* p : {(const void*)c.k, (const void*)c.v}) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (overlap(e, {lo, lo + (uintptr_t)cache_bytes(c)})) return true;
  }
  for (const void* p : {(const void*)c.k_scale, (const void*)c.v_scale}) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (overlap(e, {lo, lo + 4 * (uintptr_t)((c.num_pages - 1) * c.scale_stride + c.heads)})) return true;
  }
  return false;
}

int validate_append(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_heads* q, const sgr_heads* k,
                    const sgr_heads* v, const sgr_heads* qo, const sgr_norm_rope* nr) {
  int rc;
  if ((rc = check_cache(c)) != SGR_OK || (rc = check_batch(b)) != SGR_OK) return rc;
  if ((q == nullptr) != (qo == nullptr)) return SGR_ERR_NULL;
  if (empty(*b)) return SGR_OK;
  const int dim = c->head_dim;
  if ((rc = check_norm_rope(nr, dim)) != SGR_OK) return rc;
  if ((rc = check_heads(k, c->heads, dim, false)) != SGR_OK) return rc;
  if ((rc = check_heads(v, c->heads, dim, false)) != SGR_OK) return rc;
  if (touches_cache(*k, *c, b->tokens) || touches_cache(*v, *c, b->tokens)) return SGR_ERR_ALIAS;
  if (q) {
    if ((rc = check_heads(q, q->heads, dim, false)) != SGR_OK) return rc;
    if ((rc = check_heads(qo, q->heads, dim, true)) != SGR_OK) return rc;
    if ((rc = check_rows(*qo, b->tokens, dim)) != SGR_OK) return rc;
    if (!same_rows(*q, *qo) && heads_overlap(*q, *qo, b->tokens, dim)) return SGR_ERR_ALIAS;
    if (heads_overlap(*k, *qo, b->tokens, dim) || heads_overlap(*v, *qo, b->tokens, dim)) return SGR_ERR_ALIAS;
    if (touches_cache(*q, *c, b->tokens) || touches_cache(*qo, *c, b->tokens)) return SGR_ERR_ALIAS;
  }
  return SGR_OK;
}

int validate_attention(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_heads* q, const sgr_heads* out,
                       float scale, int window) {
  int rc;
  if ((rc = check_cache(c)) != SGR_OK || (rc = check_batch(b)) != SGR_OK) return rc;
  if (!std::isfinite(scale) || window < 0) return SGR_ERR_SHAPE;
  if (empty(*b)) return SGR_OK;
  if (!q || !out) return SGR_ERR_NULL;
  if ((rc = check_heads(q, q->heads, c->head_dim, false)) != SGR_OK) return rc;
  if (q->heads % c->heads) return SGR_ERR_SHAPE;
  if ((rc = check_heads(out, q->heads, c->head_dim, true)) != SGR_OK) return rc;
  if (q->heads / c->heads > kMaxGroup) return SGR_ERR_UNSUPPORTED;
  if ((rc = check_rows(*out, b->tokens, c->head_dim)) != SGR_OK) return rc;
  if (heads_overlap(*q, *out, b->tokens, c->head_dim)) return SGR_ERR_ALIAS;
  if (touches_cache(*out, *c, b->tokens)) return SGR_ERR_ALIAS;
  return SGR_OK;
}

// ------------------------------------------------------------ device set-up
struct KvDevice {
  std::once_flag once;
  int status = SGR_ERR_DEVICE;
  int sms = 0;
  unsigned* err = nullptr;
};
KvDevice g_kv[kMaxDevices];

int current_kv_device(KvDevice** out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SGR_ERR_DEVICE;
  }
  const int rc = sgr::kv_init_device(dev);
  if (rc == SGR_OK) *out = &g_kv[dev];
  return rc;
}

// ------------------------------------------------------------ launches
sgr::KvHeads heads_of(const sgr_heads* x) {
  if (!x) return {nullptr, 0, 0, 0};
  return {static_cast<__nv_bfloat16*>(x->data), x->token_stride, x->head_stride, x->heads};
}

sgr::NormRope norm_rope_of(const sgr_norm_rope& n) {
  return {static_cast<const __nv_bfloat16*>(n.q_weight), static_cast<const __nv_bfloat16*>(n.k_weight), n.table, n.eps,
          n.table_rows, n.table ? n.rot_dim : 0, n.interleaved};
}

sgr::KvBatch batch_of(const sgr_kv_batch& b) {
  return {b.block_table, b.seq_len, b.q_start, b.table_stride, b.batch, b.max_pages, b.tokens};
}

sgr::KvCacheRef cache_of(const sgr_kv_cache& c) {
  const int shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  return {static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.k_scale, c.v_scale, c.page_stride, c.head_stride,
          c.token_stride, c.scale_stride, c.num_pages, shift, c.heads};
}

template <class Fn, class... Params>
int launch(Fn fn, dim3 grid, int threads, size_t smem, unsigned flags, void* stream, const Params&... p) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = (flags & SGR_FLAG_NO_PDL) ? 0 : 1;
  if (cudaLaunchKernelEx(&lc, fn, p...) != cudaSuccess) {
    cudaGetLastError();
    return SGR_ERR_LAUNCH;
  }
  return SGR_OK;
}

// Passes over a row's heads of one block: one while that does not fill the
// GPU (few rows: latency), four beyond (the reads of four heads a thread are
// then under way at once, and the row's cosines, sines and weights are read
// once for them).  32 heads of 128, one pass and four: 1.6 and 2.1 us (64
// rows), 2.5 and 3.6 (256), 4.0 and 4.1 (700: the change-over), 8.0 and 6.9
// (1500); 72 heads: 15.5 and 12.7 (1500), 114 and 90 (12345).
int rope_passes(int sms, long long rows, int heads, int per_pass) {
  return rows * ((heads + per_pass - 1) / per_pass) > 16LL * sms && heads > per_pass ? 4 : 1;
}

int run_rope(const sgr_heads* q, const sgr_heads* k, const sgr_heads* qo, const sgr_heads* ko, const int* positions,
             int tokens, int dim, const sgr_norm_rope* nr, unsigned flags, void* stream) {
  int rc = validate_rope(q, k, qo, ko, positions, tokens, dim, nr);
  if (rc != SGR_OK || tokens == 0) return rc;
  KvDevice* dev;
  if ((rc = current_kv_device(&dev)) != SGR_OK) return rc;
  sgr::RopeParams p;
  p.q = heads_of(q);
  p.k = heads_of(k);
  p.qo = heads_of(qo);
  p.ko = heads_of(ko);
  p.positions = positions;
  p.nr = norm_rope_of(*nr);
  p.err = dev->err;
  const int per_pass = sgr::kRopeThreads / (dim / 8), passes = rope_passes(dev->sms, tokens, p.q.heads + p.k.heads, per_pass);
  p.heads_per_block = per_pass * passes;
  p.q_chunks = (p.q.heads + p.heads_per_block - 1) / p.heads_per_block;
  const dim3 grid(tokens, p.q_chunks + (p.k.heads + p.heads_per_block - 1) / p.heads_per_block);
  void (*fn)(const sgr::RopeParams) =
      dim == 64 ? (passes == 4 ? sgr::qk_norm_rope_kernel<64, 4> : sgr::qk_norm_rope_kernel<64, 1>)
                : (passes == 4 ? sgr::qk_norm_rope_kernel<128, 4> : sgr::qk_norm_rope_kernel<128, 1>);
  return launch(fn, grid, sgr::kRopeThreads, 0, flags, stream, p);
}

using AppendFn = void (*)(const sgr::AppendParams);

template <int D, int kQPass>
AppendFn append_fn_pass(int pass) {
  if (pass == 1) return sgr::kv_append_kernel<D, 1, kQPass>;
  if (pass == 2) return sgr::kv_append_kernel<D, 2, kQPass>;
  if (pass == 4 || D == 64) return sgr::kv_append_kernel<D, 4, kQPass>;
  return sgr::kv_append_kernel<D, D == 64 ? 4 : 8, kQPass>;
}

// The kernel whose threads hold a whole page of new tokens, or `most` of them.
AppendFn append_fn(int dim, int page_size, int most, int q_passes) {
  const int tok = sgr::kAppendThreads / (dim / 8), n = most < page_size ? most : page_size;
  const int pass = n <= tok ? 1 : n <= 2 * tok ? 2 : n <= 4 * tok ? 4 : 8;
  if (dim == 64) return q_passes == 4 ? append_fn_pass<64, 4>(pass) : append_fn_pass<64, 1>(pass);
  return q_passes == 4 ? append_fn_pass<128, 4>(pass) : append_fn_pass<128, 1>(pass);
}

int run_append(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_heads* q, const sgr_heads* k,
               const sgr_heads* v, const sgr_heads* qo, const sgr_norm_rope* nr, unsigned flags, void* stream) {
  int rc = validate_append(c, b, q, k, v, qo, nr);
  if (rc != SGR_OK || empty(*b)) return rc;
  KvDevice* dev;
  if ((rc = current_kv_device(&dev)) != SGR_OK) return rc;
  sgr::AppendParams p;
  p.q = heads_of(q);
  p.k = heads_of(k);
  p.v = heads_of(v);
  p.qo = heads_of(qo);
  p.cache = cache_of(*c);
  p.batch = batch_of(*b);
  p.nr = norm_rope_of(*nr);
  p.err = dev->err;
  // Pages written to: at most one per row; a sequence of n rows reaches at
  // most (n - 1) / page_size + 2 of them.
  long long slots = (long long)b->tokens / c->page_size + 2LL * b->batch;
  if (slots > b->tokens) slots = b->tokens;
  const int per_pass = sgr::kAppendThreads / (c->head_dim / 8);
  const int q_passes = q ? rope_passes(dev->sms, b->tokens, q->heads, per_pass) : 1;
  p.heads_per_block = per_pass * q_passes;
  p.q_chunks = q ? (q->heads + p.heads_per_block - 1) / p.heads_per_block : 0;
  const long long q_blocks = (long long)b->tokens * p.q_chunks, blocks = q_blocks + slots * c->heads * 2;
  if (blocks > 0x7fffffffLL) return SGR_ERR_UNSUPPORTED;
  p.q_blocks = (int)q_blocks;
  return launch(append_fn(c->head_dim, c->page_size, b->tokens, q_passes), dim3((unsigned)blocks), sgr::kAppendThreads, 0,
                flags, stream, p);
}

// ------------------------------------------------------------ attention
using AttnFn = void (*)(const CUtensorMap, const CUtensorMap, const sgr::AttnParams);
using JoinFn = void (*)(const sgr::AttnParams);

struct AttnKernel {
  AttnFn fn;
  JoinFn join;
  int smem, threads, join_rows;
};

template <int D, int NT>
AttnKernel attn_kernel_of() {
  return {sgr::kv_attn_kernel<D, NT>, sgr::kv_attn_join_kernel<D, NT>, sgr::attn_smem_bytes<D, NT>(),
          sgr::AttnShape<D, NT>::kThreads, sgr::JoinShape<NT>::kRows};
}

template <int D>
AttnKernel attn_rows_kernel_of() {
  return {sgr::kv_attn_rows_kernel<D>, sgr::kv_attn_join_kernel<D, sgr::kRowsNT>, sgr::rows_attn_smem_bytes<D>(),
          sgr::kRowsThreads, sgr::JoinShape<sgr::kRowsNT>::kRows};
}

template <int D>
AttnKernel attn_few_kernel(int nt) {
  return nt == 8 ? attn_kernel_of<D, 8>() : nt == 16 ? attn_kernel_of<D, 16>() : nt == 24 ? attn_kernel_of<D, 24>() : attn_kernel_of<D, 32>();
}

AttnKernel attn_kernel(int dim, int nt) {
  if (nt == sgr::kRowsNT) return dim == 64 ? attn_rows_kernel_of<64>() : attn_rows_kernel_of<128>();
  return dim == 64 ? attn_few_kernel<64>(nt) : attn_few_kernel<128>(nt);
}

struct AttnPlan {
  int nt;           // rows of a row tile
  int grid;
  bool split;       // whether a row tile may span CTAs
  bool reuse;       // whether a sequence may have several row tiles
  bool fits;        // 31 bits hold the number of units
  int64_t bytes;    // workspace
};

AttnPlan attn_plan(int sms, const sgr_kv_cache& c, const sgr_kv_batch& b, int q_heads, unsigned flags) {
  AttnPlan a;
  const long long group = q_heads / c.heads, rows = (b.max_new > 0 ? b.max_new : 1) * group;
  const long long tiles = ((long long)b.max_pages * c.page_size + sgr::kAttnTile - 1) / sgr::kAttnTile;
  auto row_tiles = [&](int nt) {  // at most
    const long long each = b.batch * ((rows + nt - 1) / nt), all = (long long)b.tokens * group / nt + b.batch;
    return c.heads * (each < all ? each : all);
  };
  // Row tiles as small as the rows of a sequence allow: the small operands and
  // accumulators are 2 and 3 nt columns wide, and so is the softmax work a tile
  // (five drafted tokens and four heads a key/value head: 29.1 us in a tile of
  // 24 against 33.9 in one of 32).
  a.nt = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : 32;
  // The 256-row kernel takes some 1.75 times (D = 64: 2.4 times) a 32-row
  // unit's time for eight times the rows, but 12 units' time to begin and end.
  // Measured with 28 heads of 128 over 4, small tiles against 256 rows: 19.1
  // and 21.4 us (8 sequences of 3000, 35 rows a head each), 122.9 and 109.8 (96
  // of them), 19.4 and 20.4 (4 of 3000, 126 rows), 51.6 and 32.6 (16 of them),
  // 24.1 and 30.9 (one, 700 rows), 84 and 47 (one, 4200 rows), 113.0 and 63.4
  // (one of 30000, 700 rows), 102.8 and 99 (32 of 9000, 63 rows), 166 and 107
  // (112 rows); 32 heads of 64 over 8: 116 and 146 (32 of 9000, 36 rows), 47.5
  // and 36.9 (3 of 20000, 96 rows).
  const double unit = c.head_dim == 64 ? 2.4 : 1.75;
  const bool gains = (double)tiles * ((double)row_tiles(32) - unit * (double)row_tiles(sgr::kRowsNT)) > 12.0 * sms;
  if ((flags & SGR_FLAG_KV_MANY_ROWS) || (gains && !(flags & SGR_FLAG_KV_FEW_ROWS))) a.nt = sgr::kRowsNT;
  // (resident CTAs)
  const long long ctas = a.nt >= 32 ? sms : 2LL * sms, items = row_tiles(a.nt);
  // Short caches are not split over CTAs: the join's launch costs more than a
  // few tiles in turn.  28 heads over 4, split and whole: 8.6 and 8.1 us (one
  // sequence of 3 tiles), 8.7 and 9.0 (of 4), 14.7 and 11.5 (64 of them), 9.6
  // and 12.6 (one of 8), 18.3 and 16.3 (64: as many row tiles as CTAs, nearly),
  // 27.4 and 29.1 (128).
  a.split = tiles > (2 * items >= ctas && items <= ctas ? 8 : 4);
  const long long units = a.split ? items * (tiles + 1) : items;
  a.fits = units < (1LL << 31) && tiles < (1 << 24);
  a.grid = (int)(units < ctas ? units : ctas);
  a.reuse = rows > a.nt;
  a.bytes = a.grid * (2LL * a.nt * (c.head_dim * 4LL + 8) + (long long)sizeof(sgr::AttnPiece));
  return a;
}

// Cache codes as a 4-D tensor (element, position in the page, head, page).
bool make_cache_tmap(CUtensorMap* m, const void* codes, const sgr_kv_cache& c) {
  sgr::detail::EncodeTiledFn fn = sgr::detail::encode_fn();
  if (!fn) return false;
  const cuuint64_t dim = (cuuint64_t)c.head_dim;
  cuuint64_t dims[4] = {dim, (cuuint64_t)c.page_size, (cuuint64_t)c.heads, (cuuint64_t)(c.num_pages ? c.num_pages : 1)};
  // (a stride that nothing is reached by may hold anything)
  cuuint64_t strides[3] = {(cuuint64_t)c.token_stride, c.heads > 1 ? (cuuint64_t)c.head_stride : dim,
                           c.num_pages > 1 ? (cuuint64_t)c.page_stride : dim};
  cuuint32_t box[4] = {(cuuint32_t)dim, (cuuint32_t)c.page_size, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(codes), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int run_attention(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_heads* q, const sgr_heads* out, float scale,
                  int window, void* workspace, int64_t workspace_bytes, unsigned flags, void* stream) {
  int rc = validate_attention(c, b, q, out, scale, window);
  if (rc != SGR_OK || empty(*b)) return rc;
  if ((flags & SGR_FLAG_KV_FEW_ROWS) && (flags & SGR_FLAG_KV_MANY_ROWS)) return SGR_ERR_UNSUPPORTED;
  if (!workspace) return SGR_ERR_NULL;
  if (!aligned(workspace, 16)) return SGR_ERR_ALIGN;
  KvDevice* dev;
  if ((rc = current_kv_device(&dev)) != SGR_OK) return rc;
  const AttnPlan a = attn_plan(dev->sms, *c, *b, q->heads, flags);
  if (!a.fits || workspace_bytes < a.bytes) return SGR_ERR_UNSUPPORTED;
  CUtensorMap tk, tv;
  // (a cache without pages: the maps are never used)
  if (!make_cache_tmap(&tk, c->num_pages ? c->k : workspace, *c) || !make_cache_tmap(&tv, c->num_pages ? c->v : workspace, *c))
    return SGR_ERR_LAUNCH;
  sgr::AttnParams p;
  p.q = heads_of(q);
  p.out = heads_of(out);
  p.cache = cache_of(*c);
  p.batch = batch_of(*b);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.window = window > 0 ? window : INT_MAX;
  p.group = q->heads / c->heads;
  p.group_inv = p.group > 1 ? (unsigned)((1ULL << 32) / p.group) : 0xffffffffu;
  p.reuse = a.reuse ? 1 : 0;
  p.whole = a.split ? 0 : 1;
  p.err = dev->err;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + 2LL * a.grid * a.nt * c->head_dim);
  p.pieces = reinterpret_cast<sgr::AttnPiece*>(p.part_ml + 2LL * a.grid * a.nt);
  const AttnKernel k = attn_kernel(c->head_dim, a.nt);
  rc = launch(k.fn, dim3(a.grid), k.threads, k.smem, flags, stream, tk, tv, p);
  if (rc != SGR_OK || !a.split) return rc;
  return launch(k.join, dim3(a.grid, a.nt / k.join_rows), sgr::kJoinThreads, 0, flags, stream, p);
}

}  // namespace

namespace sgr {

int kv_init_device(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return SGR_ERR_DEVICE;
  KvDevice& d = g_kv[dev];
  std::call_once(d.once, [&] {
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || d.sms <= 0) {
      cudaGetLastError();
      return;
    }
    int prev = -1;
    if (cudaGetDevice(&prev) != cudaSuccess || (prev != dev && cudaSetDevice(dev) != cudaSuccess)) {
      cudaGetLastError();
      return;
    }
    bool ok = true;
    for (int dim : {64, 128})
      for (int nt : {8, 16, 24, 32, sgr::kRowsNT})
        ok = ok && set_kernel_smem_attrs(reinterpret_cast<const void*>(attn_kernel(dim, nt).fn)) == cudaSuccess;
    if (prev != dev) cudaSetDevice(prev);
    if (ok)
      d.status = device_error_word(dev, &d.err);
    else
      cudaGetLastError();
  });
  return d.status;
}

}  // namespace sgr

extern "C" {

int sgr_qk_norm_rope(const sgr_heads* q, const sgr_heads* k, const sgr_heads* q_out, const sgr_heads* k_out,
                     const int* positions, int tokens, int head_dim, const sgr_norm_rope* nr, unsigned flags,
                     void* stream) {
  return run_rope(q, k, q_out, k_out, positions, tokens, head_dim, nr, flags, stream);
}

int sgr_kv_append(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const sgr_heads* k,
                  const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr, unsigned flags, void* stream) {
  return run_append(cache, batch, q, k, v, q_out, nr, flags, stream);
}

int sgr_kv_attention(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const sgr_heads* out,
                     float scale, int window, void* workspace, int64_t workspace_bytes, unsigned flags, void* stream) {
  return run_attention(cache, batch, q, out, scale, window, workspace, workspace_bytes, flags, stream);
}

int sgr_kv_attention_workspace(int device, const sgr_kv_cache* cache, const sgr_kv_batch* batch, int q_heads,
                               unsigned flags, int64_t* bytes) {
  if (!bytes) return SGR_ERR_NULL;
  int rc;
  if ((rc = check_cache(cache)) != SGR_OK || (rc = check_batch(batch)) != SGR_OK) return rc;
  if (q_heads < 1 || q_heads % cache->heads) return SGR_ERR_SHAPE;
  if ((rc = sgr::kv_init_device(device)) != SGR_OK) return rc;
  *bytes = attn_plan(g_kv[device].sms, *cache, *batch, q_heads, flags).bytes;
  return SGR_OK;
}

int sgr_validate_qk_norm_rope(const sgr_heads* q, const sgr_heads* k, const sgr_heads* q_out, const sgr_heads* k_out,
                              const int* positions, int tokens, int head_dim, const sgr_norm_rope* nr) {
  return validate_rope(q, k, q_out, k_out, positions, tokens, head_dim, nr);
}

int sgr_validate_kv_append(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                           const sgr_heads* k, const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr) {
  return validate_append(cache, batch, q, k, v, q_out, nr);
}

int sgr_validate_kv_attention(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                              const sgr_heads* out, float scale, int window) {
  return validate_attention(cache, batch, q, out, scale, window);
}

}  // extern "C"
