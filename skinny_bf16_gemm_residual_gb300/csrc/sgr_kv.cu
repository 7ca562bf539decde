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
#include "sgr_kv_evict.cuh"
#include "sgr_kv_kernels.h"

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

// n numbers of 4 bytes.
Extent words_extent(const void* p, long long n) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + 4 * (uintptr_t)(n > 0 ? n : 0)};
}

// Whether memory and the cache (codes or scales) share bytes.
bool touches_cache(Extent e, const sgr_kv_cache& c) {
  if (c.num_pages == 0) return false;
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

// Whether rows of heads and the cache (codes or scales) share memory.
bool touches_cache(const sgr_heads& x, const sgr_kv_cache& c, long long tokens) {
  return touches_cache(heads_extent(x, tokens, c.head_dim), c);
}

int validate_append(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_heads* q, const sgr_heads* k,
                    const sgr_heads* v, const sgr_heads* qo, const sgr_norm_rope* nr, const int* positions) {
  int rc;
  if ((rc = check_cache(c)) != SGR_OK || (rc = check_batch(b)) != SGR_OK) return rc;
  if ((q == nullptr) != (qo == nullptr)) return SGR_ERR_NULL;
  if (empty(*b)) return SGR_OK;
  const int dim = c->head_dim;
  if (!aligned(positions, 4)) return SGR_ERR_ALIGN;
  if ((rc = check_norm_rope(nr, dim)) != SGR_OK) return rc;
  if ((rc = check_heads(k, c->heads, dim, false)) != SGR_OK) return rc;
  if ((rc = check_heads(v, c->heads, dim, false)) != SGR_OK) return rc;
  if (touches_cache(*k, *c, b->tokens) || touches_cache(*v, *c, b->tokens)) return SGR_ERR_ALIAS;
  // (blocks write while others still read positions)
  const Extent at = words_extent(positions, positions ? b->tokens : 0);
  if (touches_cache(at, *c)) return SGR_ERR_ALIAS;
  if (q) {
    if ((rc = check_heads(q, q->heads, dim, false)) != SGR_OK) return rc;
    if ((rc = check_heads(qo, q->heads, dim, true)) != SGR_OK) return rc;
    if ((rc = check_rows(*qo, b->tokens, dim)) != SGR_OK) return rc;
    if (!same_rows(*q, *qo) && heads_overlap(*q, *qo, b->tokens, dim)) return SGR_ERR_ALIAS;
    if (heads_overlap(*k, *qo, b->tokens, dim) || heads_overlap(*v, *qo, b->tokens, dim)) return SGR_ERR_ALIAS;
    if (overlap(at, heads_extent(*qo, b->tokens, dim))) return SGR_ERR_ALIAS;
    if (touches_cache(*q, *c, b->tokens) || touches_cache(*qo, *c, b->tokens)) return SGR_ERR_ALIAS;
  }
  return SGR_OK;
}

// (NULL: no mask)
int check_mask(const sgr_kv_mask* m, const sgr_kv_batch& b) {
  if (!m) return SGR_OK;
  if (m->reserved != 0) return SGR_ERR_UNSUPPORTED;
  if (m->window < 0 || m->sinks < 0) return SGR_ERR_SHAPE;
  if (!m->tree || empty(b)) return SGR_OK;
  if (!aligned(m->tree, 8)) return SGR_ERR_ALIGN;
  if (m->tree_words < 1 || 64LL * m->tree_words < b.max_new || m->tree_stride < m->tree_words) return SGR_ERR_SHAPE;
  if (m->tree_stride > kMaxStride) return SGR_ERR_UNSUPPORTED;
  return SGR_OK;
}

// The words of a mask's trees, which are read while outputs are written.
Extent tree_extent(const sgr_kv_mask* m, const sgr_kv_batch& b) {
  if (!m || !m->tree) return {0, 0};
  return words_extent(m->tree, 2 * ((b.tokens - 1) * m->tree_stride + m->tree_words));
}

int validate_attention(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_heads* q, const sgr_heads* out,
                       const float* lse, float scale, const sgr_kv_mask* mask) {
  int rc;
  if ((rc = check_cache(c)) != SGR_OK || (rc = check_batch(b)) != SGR_OK) return rc;
  if (!std::isfinite(scale)) return SGR_ERR_SHAPE;
  if ((rc = check_mask(mask, *b)) != SGR_OK) return rc;
  if (empty(*b)) return SGR_OK;
  if (!q || !out) return SGR_ERR_NULL;
  if ((rc = check_heads(q, q->heads, c->head_dim, false)) != SGR_OK) return rc;
  if (q->heads % c->heads) return SGR_ERR_SHAPE;
  if ((rc = check_heads(out, q->heads, c->head_dim, true)) != SGR_OK) return rc;
  if (q->heads / c->heads > kMaxGroup) return SGR_ERR_UNSUPPORTED;
  if ((rc = check_rows(*out, b->tokens, c->head_dim)) != SGR_OK) return rc;
  if (heads_overlap(*q, *out, b->tokens, c->head_dim)) return SGR_ERR_ALIAS;
  if (touches_cache(*out, *c, b->tokens)) return SGR_ERR_ALIAS;
  const Extent tree = tree_extent(mask, *b);
  if (overlap(tree, heads_extent(*out, b->tokens, c->head_dim))) return SGR_ERR_ALIAS;
  if (lse) {
    if (!aligned(lse, 4)) return SGR_ERR_ALIGN;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(lse);
    const Extent e{lo, lo + 4 * (uintptr_t)b->tokens * q->heads};
    if (overlap(e, heads_extent(*q, b->tokens, c->head_dim)) || overlap(e, heads_extent(*out, b->tokens, c->head_dim)) ||
        overlap(e, tree) || touches_cache(e, *c))
      return SGR_ERR_ALIAS;
  }
  return SGR_OK;
}

// A mass for each position of a cache: positions must not overlap, nor share
// memory with the cache.
int check_masses(const sgr_kv_masses* m, const sgr_kv_cache& c, Extent* extent) {
  if (!m) return SGR_ERR_NULL;
  *extent = {0, 0};
  if (c.num_pages == 0) return SGR_OK;
  if (!m->data) return SGR_ERR_NULL;
  if (!aligned(m->data, 4)) return SGR_ERR_ALIGN;
  struct Dim {
    long long stride, count;
  } d[2] = {{m->head_stride, c.heads}, {m->page_stride, c.num_pages}};
  for (const Dim& x : d) {
    if (x.count > 1 && x.stride < 0) return SGR_ERR_SHAPE;
    if (x.stride > kMaxStride) return SGR_ERR_UNSUPPORTED;
  }
  if (d[0].stride > d[1].stride) std::swap(d[0], d[1]);
  long long span = c.page_size;
  for (const Dim& x : d)
    if (x.count > 1) {
      if (x.stride < span) return SGR_ERR_SHAPE;
      span += (x.count - 1) * x.stride;
    }
  const uintptr_t lo = reinterpret_cast<uintptr_t>(m->data);
  *extent = {lo, lo + 4 * (uintptr_t)span};
  return touches_cache(*extent, c) ? SGR_ERR_ALIAS : SGR_OK;
}

int validate_mass(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_heads* q, const float* lse,
                  const sgr_kv_masses* mass, float scale, const sgr_kv_mask* mask) {
  int rc;
  if ((rc = check_cache(c)) != SGR_OK || (rc = check_batch(b)) != SGR_OK) return rc;
  if (!std::isfinite(scale)) return SGR_ERR_SHAPE;
  if ((rc = check_mask(mask, *b)) != SGR_OK) return rc;
  if (empty(*b)) return SGR_OK;
  if (!q || !lse) return SGR_ERR_NULL;
  if ((rc = check_heads(q, q->heads, c->head_dim, false)) != SGR_OK) return rc;
  if (q->heads % c->heads) return SGR_ERR_SHAPE;
  if (q->heads / c->heads > kMaxGroup) return SGR_ERR_UNSUPPORTED;
  if (!aligned(lse, 4)) return SGR_ERR_ALIGN;
  Extent e;
  if ((rc = check_masses(mass, *c, &e)) != SGR_OK) return rc;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(lse);
  if (overlap(e, heads_extent(*q, b->tokens, c->head_dim)) || overlap(e, {lo, lo + 4 * (uintptr_t)b->tokens * q->heads}) ||
      overlap(e, tree_extent(mask, *b)))
    return SGR_ERR_ALIAS;
  return SGR_OK;
}

int validate_evict(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_kv_masses* mass, const sgr_kv_eviction* ev) {
  int rc;
  if ((rc = check_cache(c)) != SGR_OK) return rc;
  if (!b || !ev) return SGR_ERR_NULL;
  sgr_kv_batch only = *b;  // (its rows do not matter)
  only.q_start = nullptr;
  only.tokens = only.batch;
  only.max_new = 1;
  if ((rc = check_batch(&only)) != SGR_OK) return rc;
  if (ev->reserved != 0) return SGR_ERR_UNSUPPORTED;
  if (ev->first < 0 || ev->recent < 0 || ev->max_pages < 0) return SGR_ERR_SHAPE;
  if (ev->max_pages > (1 << 24)) return SGR_ERR_UNSUPPORTED;
  if (b->batch == 0) return SGR_OK;
  if (!ev->keep || !ev->new_len || (ev->max_pages > 0 && (!ev->table || !ev->kept))) return SGR_ERR_NULL;
  if (!aligned(ev->keep, 4) || !aligned(ev->new_len, 4) || !aligned(ev->table, 4) || !aligned(ev->kept, 4))
    return SGR_ERR_ALIGN;
  if (ev->table_stride < ev->max_pages) return SGR_ERR_SHAPE;
  if (ev->table_stride > kMaxStride) return SGR_ERR_UNSUPPORTED;
  Extent e[3];  // what is written: masses, positions, lengths
  if ((rc = check_masses(mass, *c, &e[0])) != SGR_OK) return rc;
  const long long rows = b->batch - 1;
  e[1] = words_extent(ev->kept, (long long)b->batch * c->heads * ev->max_pages * c->page_size);
  e[2] = words_extent(ev->new_len, b->batch);
  const Extent in[4] = {words_extent(b->seq_len, b->batch), words_extent(ev->keep, b->batch),
                        words_extent(b->block_table, b->max_pages > 0 ? rows * b->table_stride + b->max_pages : 0),
                        words_extent(ev->table, ev->max_pages > 0 ? rows * ev->table_stride + ev->max_pages : 0)};
  for (int i = 0; i < 3; ++i) {
    for (const Extent& x : in)
      if (overlap(e[i], x)) return SGR_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(e[i], e[j])) return SGR_ERR_ALIAS;
    if (touches_cache(e[i], *c)) return SGR_ERR_ALIAS;
  }
  for (const Extent& x : in)
    if (touches_cache(x, *c)) return SGR_ERR_ALIAS;
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
               const sgr_heads* v, const sgr_heads* qo, const sgr_norm_rope* nr, const int* positions, unsigned flags,
               void* stream) {
  int rc = validate_append(c, b, q, k, v, qo, nr, positions);
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
  p.positions = nr->table ? positions : nullptr;
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
sgr::AttnKernel attn_kernel(int dim, int nt, bool masked) {
  if (masked) return sgr::attn_kernel_masked(dim, nt);
  return dim == 64 ? sgr::attn_kernel_of<64, false>(nt) : sgr::attn_kernel_of<128, false>(nt);
}

struct Join {
  sgr::JoinFn fn;
  int rows;  // of a block
};

template <int D>
Join join_kernel(int nt) {
  switch (nt) {
    case 8: return {sgr::kv_attn_join_kernel<D, 8>, sgr::JoinShape<8>::kRows};
    case 16: return {sgr::kv_attn_join_kernel<D, 16>, sgr::JoinShape<16>::kRows};
    case 24: return {sgr::kv_attn_join_kernel<D, 24>, sgr::JoinShape<24>::kRows};
    case 32: return {sgr::kv_attn_join_kernel<D, 32>, sgr::JoinShape<32>::kRows};
    default: return {sgr::kv_attn_rows_join_kernel<D>, 32 * (sgr::kRowsJoinThreads / 32 / (D / 16))};
  }
}

struct AttnPlan {
  int nt;           // rows of a row tile
  int grid;
  bool split;       // whether a row tile may span CTAs
  bool reuse;       // whether a sequence may have several row tiles
  bool fits;        // 31 bits hold the number of units
  int64_t bytes;    // workspace
  int64_t any_window;  // workspace for the same sizes under any window
};

AttnPlan attn_plan(int sms, const sgr_kv_cache& c, const sgr_kv_batch& b, int q_heads, unsigned flags,
                   const sgr_kv_mask& mask) {
  AttnPlan a;
  const long long group = q_heads / c.heads, rows = (b.max_new > 0 ? b.max_new : 1) * group;
  const long long table_tiles = ((long long)b.max_pages * c.page_size + sgr::kAttnTile - 1) / sgr::kAttnTile;
  long long tiles = table_tiles;
  if (mask.window > 0) {
    const long long seen = ((long long)mask.window + b.max_new) / sgr::kAttnTile + 2 + (mask.sinks + sgr::kAttnTile - 1LL) / sgr::kAttnTile;
    if (seen < tiles) tiles = seen;
  }
  auto row_tiles = [&](int nt) {  // at most
    const long long each = b.batch * ((rows + nt - 1) / nt), all = (long long)b.tokens * group / nt + b.batch;
    return c.heads * (each < all ? each : all);
  };
  // Row tiles as small as the rows of a sequence allow: the small operands and
  // accumulators are 2 and 3 nt columns wide, and so is the softmax work a tile
  // (five drafted tokens and four heads a key/value head: 29.1 us in a tile of
  // 24 against 33.9 in one of 32).
  a.nt = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : 32;
  // Work that does not fill the GPU even in smaller row tiles takes those: more
  // CTAs, each with less (7 drafted tokens of 7 heads a key/value head over 700).
  for (int nt : {8, 16, 24})
    if (nt < a.nt && row_tiles(nt) * (tiles + 1) <= 2LL * sms) {
      a.nt = nt;
      break;
    }
  // The 256-row kernel takes some 1.25 times a 32-row unit's time for eight times
  // the rows, but some 8 units' time to begin and end.  Measured, small tiles against
  // 256 rows, one sequence of the length and the others of 1 to it, 28 heads of 128
  // over 4: 118 and 96 us (96 of 3000, 35 rows a head each), 22.4 and 23.7 (4 of
  // 3000, 126 rows), 57 and 31 (16 of 3000, 126 rows), 34 and 26 (8 of 4000, 112
  // rows), 25.2 and 27.7 (one of 2000, 700 rows), 117 and 57 (one of 30000, 448
  // rows), 211 and 92 (32 of 9000, 112 rows; 306 and 133 where all are 9000 long),
  // 64 and 52 (64 of 1500, 63 rows), but also 30.8 and 28.8 (24 of 1500, 63 rows);
  // 32 heads of 64 over 8: 57 and 41 (16 of 5000, 48 rows), 178 and 134 (32 of 9000,
  // 36 rows; 285 and 220 where all are 9000 long), 24.3 and 19.9 (4 of 1500, 160
  // rows), 54 and 37 (3 of 20000, 96 rows).
  // It also sees a query's small elements in fewer bits (sgr_attention.h).  Calls
  // over all positions up to a row's own, or the last of them, keep the few-row
  // kernel's longer, whatever their window, at up to a third of the speed: rows of
  // 36 to 64 in the figures above, and the 160 rows.  (So a log-sum-exp changes no
  // output.)  Of those that do not, short windows take the few-row kernel: 15.4 and
  // 15.7 us (8 of 4000, 112 rows, window 256: gain 2.3), 19.4 and 21.1 (one of 30000,
  // 448 rows, 1024: 3.0), but 23.3 and 18.9 (8 of 4000, 1024: 5.8), 32 and 24 (16 of
  // 3000, 126 rows, 512: 6.9), 31 and 33 (one of 30000, 4096: 10), 50 and 24 (32 of
  // 9000, 112 rows, 512: 14).
  const bool plain = !mask.tree && !(mask.window > 0 && mask.sinks > 0);
  auto gain = [&](long long t, double unit) {  // 32-row units that an SM saves
    return (double)t * ((double)row_tiles(32) - unit * (double)row_tiles(sgr::kRowsNT)) / sms;
  };
  const bool gains = plain ? gain(table_tiles, c.head_dim == 64 ? 2.4 : 1.75) > 12.0 && gain(tiles, 1.25) > 5.0
                           : gain(tiles, 1.25) > 8.0;
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
  auto bytes = [&](long long grid, int nt) { return grid * (2LL * nt * (c.head_dim * 4LL + 8) + (long long)sizeof(sgr::AttnPiece)); };
  a.bytes = a.any_window = bytes(a.grid, a.nt);
  for (int nt : {8, 16, 24, 32}) {
    const long long most = row_tiles(nt) * (tiles + 1), held = nt >= 32 ? sms : 2LL * sms;
    const int64_t need = bytes(most < held ? most : held, nt);
    if (nt < a.nt && need > a.any_window) a.any_window = need;
  }
  return a;
}

// The workspace depends on the sizes alone and is enough for any mask: with a
// tree or without, and with windows, which make the tiles of a sequence fewer,
// and by that perhaps the row tiles smaller, of which more are under way.
int64_t attn_workspace(int sms, const sgr_kv_cache& c, const sgr_kv_batch& b, int q_heads, unsigned flags) {
  sgr_kv_mask mask = {};
  const int64_t plain = attn_plan(sms, c, b, q_heads, flags, mask).any_window;
  const uint64_t some = 0;
  mask.tree = &some;  // (not looked at)
  const int64_t tree = attn_plan(sms, c, b, q_heads, flags, mask).any_window;
  return plain > tree ? plain : tree;
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

// What the walk of the work and the masks need, of any operator over the cache.
void attn_params(sgr::AttnParams* p, const sgr_kv_cache& c, const sgr_kv_batch& b, const sgr_heads& q, float scale,
                 const sgr_kv_mask* mask, unsigned* err) {
  p->q = heads_of(&q);
  p->cache = cache_of(c);
  p->batch = batch_of(b);
  p->scale_log2 = scale * 1.4426950408889634f;
  const sgr_kv_mask m = mask ? *mask : sgr_kv_mask{};
  p->window = m.window > 0 ? m.window : INT_MAX;
  p->sinks = m.window > 0 ? m.sinks : 0;
  p->tree = reinterpret_cast<const unsigned long long*>(m.tree);
  p->tree_stride = m.tree_stride;
  p->tree_words = m.tree_words;
  p->group = q.heads / c.heads;
  p->group_inv = p->group > 1 ? (unsigned)((1ULL << 32) / p->group) : 0xffffffffu;
  p->err = err;
}

sgr_kv_mask windowed(int window) {
  sgr_kv_mask m = {};
  m.window = window;
  return m;
}

int run_attention(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_heads* q, const sgr_heads* out, float* lse,
                  float scale, const sgr_kv_mask* mask, void* workspace, int64_t workspace_bytes, unsigned flags,
                  void* stream) {
  int rc = validate_attention(c, b, q, out, lse, scale, mask);
  if (rc != SGR_OK || empty(*b)) return rc;
  if ((flags & SGR_FLAG_KV_FEW_ROWS) && (flags & SGR_FLAG_KV_MANY_ROWS)) return SGR_ERR_UNSUPPORTED;
  if (!workspace) return SGR_ERR_NULL;
  if (!aligned(workspace, 16)) return SGR_ERR_ALIGN;
  KvDevice* dev;
  if ((rc = current_kv_device(&dev)) != SGR_OK) return rc;
  const AttnPlan a = attn_plan(dev->sms, *c, *b, q->heads, flags, mask ? *mask : sgr_kv_mask{});
  if (!a.fits || workspace_bytes < a.bytes) return SGR_ERR_UNSUPPORTED;
  CUtensorMap tk, tv;
  // (a cache without pages: the maps are never used)
  if (!make_cache_tmap(&tk, c->num_pages ? c->k : workspace, *c) || !make_cache_tmap(&tv, c->num_pages ? c->v : workspace, *c))
    return SGR_ERR_LAUNCH;
  sgr::AttnParams p;
  attn_params(&p, *c, *b, *q, scale, mask, dev->err);
  p.out = heads_of(out);
  p.lse = lse;
  p.reuse = a.reuse ? 1 : 0;
  p.whole = a.split ? 0 : 1;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + 2LL * a.grid * a.nt * c->head_dim);
  p.pieces = reinterpret_cast<sgr::AttnPiece*>(p.part_ml + 2LL * a.grid * a.nt);
  const sgr::AttnKernel k = attn_kernel(c->head_dim, a.nt, p.sinks > 0 || p.tree || p.lse);
  rc = launch(k.fn, dim3(a.grid), k.threads, k.smem, flags, stream, tk, tv, p);
  if (rc != SGR_OK || !a.split) return rc;
  const Join join = c->head_dim == 64 ? join_kernel<64>(a.nt) : join_kernel<128>(a.nt);
  return launch(join.fn, dim3(a.grid, a.nt / join.rows), sgr::kJoinThreads, 0, flags, stream, p);
}

// ------------------------------------------------------------ mass
struct MassPlan {
  int nt;         // rows of a row tile
  int grid;
  int tiles;      // of keys, of a sequence
  bool part;      // whether a sequence may have several row tiles
  bool fits;
  int64_t bytes;  // workspace
};

MassPlan mass_plan(int sms, const sgr_kv_cache& c, const sgr_kv_batch& b, int q_heads) {
  MassPlan m;
  const long long group = q_heads / c.heads, rows = (b.max_new > 0 ? b.max_new : 1) * group;
  m.nt = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : sgr::kMassRows;
  m.part = rows > m.nt;
  const long long tiles = ((long long)b.max_pages * c.page_size + sgr::kAttnTile - 1) / sgr::kAttnTile;
  const long long row_tiles = m.part ? (long long)b.tokens * group / m.nt + b.batch : b.batch;  // at most
  const long long units = c.heads * row_tiles * (tiles + 1);
  m.fits = units < (1LL << 31) && tiles < (1 << 24) && (!m.part || b.batch <= 65535);
  m.tiles = (int)tiles;
  m.grid = (int)(units < 2LL * sms ? units : 2LL * sms);
  m.bytes = m.part && m.fits ? row_tiles * c.heads * tiles * sgr::kAttnTile * 4LL : 0;
  return m;
}

int run_mass(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_heads* q, const float* lse,
             const sgr_kv_masses* mass, float scale, const sgr_kv_mask* mask, void* workspace, int64_t workspace_bytes,
             unsigned flags, void* stream) {
  int rc = validate_mass(c, b, q, lse, mass, scale, mask);
  if (rc != SGR_OK || empty(*b)) return rc;
  KvDevice* dev;
  if ((rc = current_kv_device(&dev)) != SGR_OK) return rc;
  const MassPlan m = mass_plan(dev->sms, *c, *b, q->heads);
  if (!m.fits) return SGR_ERR_UNSUPPORTED;
  if (m.part) {
    if (!workspace) return SGR_ERR_NULL;
    if (!aligned(workspace, 16)) return SGR_ERR_ALIGN;
    if (workspace_bytes < m.bytes) return SGR_ERR_UNSUPPORTED;
  }
  if (c->num_pages == 0 || m.tiles == 0) return SGR_OK;  // (no position has a place)
  CUtensorMap tk;
  if (!make_cache_tmap(&tk, c->k, *c)) return SGR_ERR_LAUNCH;
  sgr::MassParams p = {};
  attn_params(&p.a, *c, *b, *q, scale, mask, dev->err);
  p.a.lse = const_cast<float*>(lse);
  p.a.reuse = m.part ? 1 : 0;
  p.mass = mass->data;
  p.page_stride = mass->page_stride;
  p.head_stride = mass->head_stride;
  p.part = m.part ? static_cast<float*>(workspace) : nullptr;
  p.tiles = m.tiles;
  p.max_new = b->max_new;
  const sgr::MassKernel k = sgr::mass_kernel(c->head_dim, m.nt);
  rc = launch(k.fn, dim3(m.grid), k.threads, k.smem, flags, stream, tk, p);
  if (rc != SGR_OK || !m.part) return rc;
  return launch(sgr::mass_join_kernel(), dim3(m.tiles, c->heads, b->batch), sgr::kAttnTile, 0, flags, stream, p);
}

// ------------------------------------------------------------ eviction
int run_evict(const sgr_kv_cache* c, const sgr_kv_batch* b, const sgr_kv_masses* mass, const sgr_kv_eviction* ev,
              unsigned flags, void* stream) {
  int rc = validate_evict(c, b, mass, ev);
  if (rc != SGR_OK || b->batch == 0) return rc;
  KvDevice* dev;
  if ((rc = current_kv_device(&dev)) != SGR_OK) return rc;
  // CTAs of a cluster: as many as hold a sequence's keys in shared memory, and
  // more while the clusters do not fill the GPU.
  const long long items = (long long)b->batch * c->heads, longest = (long long)b->max_pages * c->page_size;
  int cluster = 1;
  while (cluster < sgr::kSelectCluster &&
         (longest > (long long)cluster * sgr::kSelectCached || (items * cluster < dev->sms && longest > cluster * 2048LL)))
    cluster *= 2;
  // Warps of the move: 16-byte runs of a page's head, two (the smallest) or four
  // a lane, eight warps a block.
  const int runs = c->page_size * c->head_dim / 16, vec = runs / 32 < 4 ? 2 : 4, warps = runs / (32 * vec);
  const int per_block = sgr::kMoveThreads / 32 / warps;
  const long long moves = (items * ev->max_pages + per_block - 1) / per_block;
  if (items * cluster > 0x7fffffffLL || items * (long long)ev->max_pages > 0x7fffff00LL)
    return SGR_ERR_UNSUPPORTED;  // (31 bits hold a block's pages, too)
  sgr::EvictParams p;
  p.cache = cache_of(*c);
  p.batch = batch_of(*b);
  if (c->num_pages == 0) p.batch.max_pages = 0;  // (no position has a place)
  p.mass = mass->data;
  p.page_stride = mass->page_stride;
  p.head_stride = mass->head_stride;
  p.keep = ev->keep;
  p.new_table = ev->table;
  p.new_stride = ev->table_stride;
  p.new_pages = ev->max_pages;
  p.first = ev->first;
  p.recent = ev->recent;
  p.kept = ev->kept;
  p.new_len = ev->new_len;
  const long long run = ((longest + cluster - 1) / cluster + 3) & ~3LL;  // of a CTA, at most
  p.cached = (int)(run < sgr::kSelectCached ? run : sgr::kSelectCached);
  p.pages_inv = ev->max_pages > 1 ? (unsigned)((1ULL << 32) / ev->max_pages) : 0xffffffffu;
  p.heads_inv = c->heads > 1 ? (unsigned)((1ULL << 32) / c->heads) : 0xffffffffu;
  p.wide = aligned(mass->data, 16) && mass->page_stride % 4 == 0 && mass->head_stride % 4 == 0;
  p.err = dev->err;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(items * cluster));
  lc.blockDim = dim3(sgr::kSelectThreads);
  lc.dynamicSmemBytes = sizeof(sgr::SelectCtl) + 4 * (size_t)p.cached;
  lc.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = (flags & SGR_FLAG_NO_PDL) ? 1 : 2;
  if (cudaLaunchKernelEx(&lc, sgr::kv_select_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return SGR_ERR_LAUNCH;
  }
  if (moves == 0) return SGR_OK;
  void (*move)(const sgr::EvictParams) = c->head_dim == 128 ? sgr::kv_move_kernel<128, 4>
                                         : vec == 2         ? sgr::kv_move_kernel<64, 2>
                                                            : sgr::kv_move_kernel<64, 4>;
  return launch(move, dim3((unsigned)moves), sgr::kMoveThreads, 0, flags, stream, p);
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
        for (bool masked : {false, true})
          ok = ok && set_kernel_smem_attrs(reinterpret_cast<const void*>(attn_kernel(dim, nt, masked).fn)) == cudaSuccess;
    for (int dim : {64, 128})
      for (int nt : {8, 16, 32, sgr::kMassRows})
        ok = ok && set_kernel_smem_attrs(reinterpret_cast<const void*>(mass_kernel(dim, nt).fn)) == cudaSuccess;
    ok = ok && set_kernel_smem_attrs(reinterpret_cast<const void*>(kv_select_kernel)) == cudaSuccess;
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
  return run_append(cache, batch, q, k, v, q_out, nr, nullptr, flags, stream);
}

int sgr_kv_append_at(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const sgr_heads* k,
                     const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr, const int* positions,
                     unsigned flags, void* stream) {
  return run_append(cache, batch, q, k, v, q_out, nr, positions, flags, stream);
}

int sgr_kv_attention(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const sgr_heads* out,
                     float scale, int window, void* workspace, int64_t workspace_bytes, unsigned flags, void* stream) {
  const sgr_kv_mask mask = windowed(window);
  return run_attention(cache, batch, q, out, nullptr, scale, &mask, workspace, workspace_bytes, flags, stream);
}

int sgr_kv_attention_masked(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                            const sgr_heads* out, float* lse, float scale, const sgr_kv_mask* mask, void* workspace,
                            int64_t workspace_bytes, unsigned flags, void* stream) {
  return run_attention(cache, batch, q, out, lse, scale, mask, workspace, workspace_bytes, flags, stream);
}

int sgr_kv_attention_workspace(int device, const sgr_kv_cache* cache, const sgr_kv_batch* batch, int q_heads,
                               unsigned flags, int64_t* bytes) {
  if (!bytes) return SGR_ERR_NULL;
  int rc;
  if ((rc = check_cache(cache)) != SGR_OK || (rc = check_batch(batch)) != SGR_OK) return rc;
  if (q_heads < 1 || q_heads % cache->heads) return SGR_ERR_SHAPE;
  if ((rc = sgr::kv_init_device(device)) != SGR_OK) return rc;
  *bytes = attn_workspace(g_kv[device].sms, *cache, *batch, q_heads, flags);
  return SGR_OK;
}

int sgr_kv_mass(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const float* lse,
                const sgr_kv_masses* mass, float scale, const sgr_kv_mask* mask, void* workspace,
                int64_t workspace_bytes, unsigned flags, void* stream) {
  return run_mass(cache, batch, q, lse, mass, scale, mask, workspace, workspace_bytes, flags, stream);
}

int sgr_kv_mass_workspace(const sgr_kv_cache* cache, const sgr_kv_batch* batch, int q_heads, int64_t* bytes) {
  if (!bytes) return SGR_ERR_NULL;
  int rc;
  if ((rc = check_cache(cache)) != SGR_OK || (rc = check_batch(batch)) != SGR_OK) return rc;
  if (q_heads < 1 || q_heads % cache->heads) return SGR_ERR_SHAPE;
  // (as the call: what it refuses might not fit 64 bits)
  if (q_heads > kMaxHeads || q_heads / cache->heads > kMaxGroup) return SGR_ERR_UNSUPPORTED;
  const MassPlan m = mass_plan(1, *cache, *batch, q_heads);
  if (!m.fits && !empty(*batch)) return SGR_ERR_UNSUPPORTED;
  *bytes = m.bytes;
  return SGR_OK;
}

int sgr_kv_evict(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_kv_masses* mass,
                 const sgr_kv_eviction* eviction, unsigned flags, void* stream) {
  return run_evict(cache, batch, mass, eviction, flags, stream);
}

int sgr_validate_kv_mass(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const float* lse,
                         const sgr_kv_masses* mass, float scale, const sgr_kv_mask* mask) {
  return validate_mass(cache, batch, q, lse, mass, scale, mask);
}

int sgr_validate_kv_evict(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_kv_masses* mass,
                          const sgr_kv_eviction* eviction) {
  return validate_evict(cache, batch, mass, eviction);
}

int sgr_validate_qk_norm_rope(const sgr_heads* q, const sgr_heads* k, const sgr_heads* q_out, const sgr_heads* k_out,
                              const int* positions, int tokens, int head_dim, const sgr_norm_rope* nr) {
  return validate_rope(q, k, q_out, k_out, positions, tokens, head_dim, nr);
}

int sgr_validate_kv_append(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                           const sgr_heads* k, const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr) {
  return validate_append(cache, batch, q, k, v, q_out, nr, nullptr);
}

int sgr_validate_kv_append_at(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                              const sgr_heads* k, const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr,
                              const int* positions) {
  return validate_append(cache, batch, q, k, v, q_out, nr, positions);
}

int sgr_validate_kv_attention(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                              const sgr_heads* out, float scale, int window) {
  const sgr_kv_mask mask = windowed(window);
  return validate_attention(cache, batch, q, out, nullptr, scale, &mask);
}

int sgr_validate_kv_attention_masked(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                                     const sgr_heads* out, const float* lse, float scale, const sgr_kv_mask* mask) {
  return validate_attention(cache, batch, q, out, lse, scale, mask);
}

}  // extern "C"
