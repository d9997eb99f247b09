// C-ABI entry points of the attention calls (declared in include/woq.h): argument checks, the
// device check and dispatch to the kernel launchers. Nothing here allocates or synchronises.
#include <algorithm>
#include <cstdint>

#include "woq.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kMaxSequences = 1 << 16;  // a tile is looked up among them in a millisecond at most
constexpr int kMaxGroup = 64;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The kernels take it times log2(e).
bool good_scale(float scale) { return scale > 0.0f && scale <= 0x1p127f; }

int64_t size_of(int32_t dtype) { return dtype == WOQ_F32 ? 4 : 2; }

int check_rows(const woq_rows *r, int64_t rows, int64_t heads, int64_t dim) {
  if (!r || (rows > 0 && !r->data)) return WOQ_EINVAL;
  if (r->dtype != WOQ_F32 && r->dtype != WOQ_F16 && r->dtype != WOQ_BF16) return WOQ_EINVAL;
  if (r->heads != heads) return WOQ_EINVAL;
  const int64_t size = size_of(r->dtype), unit = 16 / size, most = (int64_t(1) << 40) / size;
  // strides below 2^40 bytes, which a tensor map holds, and an array within 2^62: its offsets fit 64 bits
  if (r->row_stride <= 0 || r->head_stride < dim || r->row_stride >= most || r->head_stride >= most ||
      r->row_stride % unit || r->head_stride % unit)
    return WOQ_ESHAPE;
  const __int128 bytes = (static_cast<__int128>(rows - 1) * r->row_stride + (heads - 1) * r->head_stride + dim) * size;
  if (rows > 0 && bytes > (__int128(1) << 62)) return WOQ_ESHAPE;
  return aligned(r->data, 16) ? WOQ_OK : WOQ_EALIGN;
}

int check_cache(const woq_kv4 *c) {
  if (!c || !c->codes || !c->scales) return WOQ_EINVAL;
  if (c->page < 16 || c->page > 65536 || (c->page & (c->page - 1))) return WOQ_EINVAL;
  if (c->dim != 64 && c->dim != 128) return WOQ_ESHAPE;
  if (c->kv_heads < 1 || c->kv_heads > 1024 || c->pages < 1 || c->pages > INT32_MAX) return WOQ_ESHAPE;
  return aligned(c->codes, 64) && aligned(c->scales, 64) ? WOQ_OK : WOQ_EALIGN;
}

int check_table(int32_t batch, const int32_t *table, int64_t width) {
  if (!table || batch < 1 || batch > kKv4MaxBatch) return WOQ_EINVAL;
  if (width < 1 || width > INT32_MAX) return WOQ_ESHAPE;
  return aligned(table, 4) ? WOQ_OK : WOQ_EALIGN;
}

// An array that is written (it passed check_rows): no two rows of heads share an element.
int check_written(const woq_rows *r, int64_t rows, int64_t dim) {
  const int64_t row = r->row_stride, head = r->head_stride, heads = r->heads;
  if (rows <= 1) return WOQ_OK;
  if (row < dim) return WOQ_ESHAPE;
  if (row >= (heads - 1) * head + dim || head >= (rows - 1) * row + dim) return WOQ_OK;  // one within the other
  for (int64_t h = 1; h < heads; ++h) {  // the two rows that lie next to h heads on
    const int64_t i = h * head / row, before = h * head - i * row;
    if ((i < rows && before < dim) || (i + 1 < rows && row - before < dim)) return WOQ_ESHAPE;
  }
  return WOQ_OK;
}

// First and one past the last byte of [rows, heads, dim].
struct Span {
  uintptr_t first, last;
};
Span span(const woq_rows &r, int64_t rows, int64_t dim) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(r.data);
  const int64_t last = (rows - 1) * r.row_stride + (r.heads - 1) * r.head_stride + dim;
  return {p, p + static_cast<uintptr_t>(last * size_of(r.dtype))};
}

// Whether an output shares bytes with another array. Slices of one fused array interleave without sharing
// any: they are compared within one row of all heads, within one head of all rows, and within one row of a
// head, wherever both arrays repeat at the same distance.
bool overlap(const woq_rows &a, const woq_rows &b, int64_t rows, int64_t dim) {
  const Span x = span(a, rows, dim), y = span(b, rows, dim);
  if (x.last <= y.first || y.last <= x.first) return false;
  const int64_t size = size_of(a.dtype);
  if (size != size_of(b.dtype)) return true;
  // b starts d bytes into a period of a: apart if that is behind a's bytes and b's end before the next period
  auto apart = [&](int64_t period, int64_t in_a, int64_t in_b) {
    const uintptr_t p = static_cast<uintptr_t>(period * size);
    const uintptr_t d = x.first <= y.first ? (y.first - x.first) % p : p - (x.first - y.first) % p;
    return d % p >= static_cast<uintptr_t>(in_a * size) && d % p + static_cast<uintptr_t>(in_b * size) <= p;
  };
  const int64_t row = a.row_stride, head = a.head_stride;
  const bool same_rows = row == b.row_stride, same_heads = head == b.head_stride;
  if (same_rows && apart(row, (a.heads - 1) * head + dim, (b.heads - 1) * b.head_stride + dim)) return false;
  if (same_heads && apart(head, (rows - 1) * row + dim, (rows - 1) * b.row_stride + dim)) return false;
  if (same_rows && same_heads && (row % head == 0 || head % row == 0) && apart(std::min(row, head), dim, dim))
    return false;
  return true;
}

// Whether an array shares bytes with the cache.
bool on_cache(const woq_rows &r, int64_t rows, const woq_kv4 &c) {
  const Span x = span(r, rows, c.dim);
  const __int128 tokens = static_cast<__int128>(c.pages) * c.kv_heads * c.page;
  auto on = [&](const void *p, __int128 bytes) {
    const uintptr_t first = reinterpret_cast<uintptr_t>(p);
    return x.first < first + bytes && first < x.last;
  };
  return on(c.codes, tokens * c.dim) || on(c.scales, tokens * (c.dim / 8));
}

int check_step(const woq_kv4 *cache, const woq_rows *k, const woq_rows *v, int64_t tokens, const int32_t *cu,
               const int32_t *start, int32_t batch, const int32_t *table, int64_t width) {
  int rc = check_cache(cache);
  if (rc != WOQ_OK) return rc;
  rc = check_table(batch, table, width);
  if (rc != WOQ_OK) return rc;
  if (!cu || tokens < 0) return WOQ_EINVAL;
  if (tokens > INT32_MAX) return WOQ_ESHAPE;
  if (!aligned(cu, 4) || !aligned(start, 4)) return WOQ_EALIGN;
  rc = check_rows(k, tokens, cache->kv_heads, cache->dim);
  if (rc != WOQ_OK) return rc;
  rc = check_rows(v, tokens, cache->kv_heads, cache->dim);
  if (rc != WOQ_OK) return rc;
  // pairs of heads, 32 of them a block at most
  return tokens * ((cache->kv_heads + 1) / 2) > (int64_t(INT32_MAX) << 5) ? WOQ_ESHAPE : WOQ_OK;
}

int step(const woq_kv4 *cache, const woq_rows *k, const woq_rows *v, int64_t tokens, const int32_t *cu,
         const int32_t *start, int32_t batch, const int32_t *table, int64_t width, bool append, void *stream) {
  int rc = check_step(cache, k, v, tokens, cu, start, batch, table, width);
  if (rc != WOQ_OK) return rc;
  if (!append && tokens > 0) {
    rc = check_written(k, tokens, cache->dim);
    if (rc != WOQ_OK) return rc;
    rc = check_written(v, tokens, cache->dim);
    if (rc != WOQ_OK) return rc;
    if (overlap(*k, *v, tokens, cache->dim) || on_cache(*k, tokens, *cache) || on_cache(*v, tokens, *cache))
      return WOQ_EINVAL;
  }
  DevInfo dev;
  rc = current_device(&dev);
  if (rc != WOQ_OK || tokens == 0) return rc;
  return launch_kv4_rows(*cache, *k, *v, tokens, cu, start, batch, table, width, append,
                         static_cast<cudaStream_t>(stream), dev);
}

}  // namespace
}  // namespace woq

using woq::DevInfo;

extern "C" {

int kv4_append(const woq_kv4 *cache, const woq_rows *k, const woq_rows *v, int64_t tokens, const int32_t *cu,
               const int32_t *start, int32_t batch, const int32_t *table, int64_t width, void *stream) {
  return woq::step(cache, k, v, tokens, cu, start, batch, table, width, true, stream);
}

int kv4_gather(const woq_kv4 *cache, const int32_t *cu, const int32_t *start, int32_t batch, const int32_t *table,
               int64_t width, int64_t tokens, const woq_rows *k, const woq_rows *v, void *stream) {
  return woq::step(cache, k, v, tokens, cu, start, batch, table, width, false, stream);
}

size_t kv4_attn_workspace_bytes(const woq_kv4 *cache, int32_t q_heads, int32_t batch) {
  if (woq::check_cache(cache) != WOQ_OK || batch < 1 || batch > woq::kKv4MaxBatch) return 0;
  if (q_heads < 1 || q_heads % cache->kv_heads || q_heads / cache->kv_heads > woq::kMaxGroup) return 0;
  DevInfo dev;
  const int sms = woq::current_device(&dev) == WOQ_OK ? dev.sm_count : 148;
  return woq::kv4_attn_workspace(batch, cache->kv_heads, q_heads / cache->kv_heads, sms);
}

int kv4_attn(const woq_rows *q, const woq_kv4 *cache, const int32_t *lens, int32_t batch, const int32_t *table,
             int64_t width, float scale, const woq_rows *o, void *workspace, size_t workspace_bytes,
             void *stream) {
  int rc = woq::check_cache(cache);
  if (rc != WOQ_OK) return rc;
  rc = woq::check_table(batch, table, width);
  if (rc != WOQ_OK) return rc;
  if (!q || !o || !lens) return WOQ_EINVAL;
  if (q->heads < 1 || q->heads % cache->kv_heads || q->heads / cache->kv_heads > woq::kMaxGroup) return WOQ_EINVAL;
  rc = woq::check_rows(q, batch, q->heads, cache->dim);
  if (rc != WOQ_OK) return rc;
  rc = woq::check_rows(o, batch, q->heads, cache->dim);
  if (rc != WOQ_OK) return rc;
  rc = woq::check_written(o, batch, cache->dim);
  if (rc != WOQ_OK) return rc;
  if (o->dtype != q->dtype || !woq::good_scale(scale)) return WOQ_EINVAL;
  if (!woq::aligned(lens, 4)) return WOQ_EALIGN;
  if (woq::overlap(*q, *o, batch, cache->dim)) return WOQ_EINVAL;
  DevInfo dev;
  rc = woq::current_device(&dev);
  const size_t need = woq::kv4_attn_workspace(batch, cache->kv_heads, q->heads / cache->kv_heads,
                                              rc == WOQ_OK ? dev.sm_count : 148);
  if (!workspace || workspace_bytes < need) return WOQ_EWORKSPACE;
  if (!woq::aligned(workspace, 256)) return WOQ_EALIGN;
  if (woq::on_cache(*o, batch, *cache)) return WOQ_EINVAL;
  if (rc != WOQ_OK) return rc;
  return woq::launch_kv4_attn(*q, *cache, lens, batch, table, width, scale, *o, workspace,
                              static_cast<cudaStream_t>(stream), dev);
}

static bool prompt_heads(int32_t q_heads, int32_t kv_heads) {
  return kv_heads >= 1 && kv_heads <= 1024 && q_heads >= 1 && q_heads <= 32768 && q_heads % kv_heads == 0;
}

size_t attn_prompt_workspace_bytes(int64_t tokens, int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t dim,
                                   int32_t dtype) {
  if (tokens < 0 || tokens > INT32_MAX || batch < 1 || batch > woq::kMaxSequences) return 0;
  if (!prompt_heads(q_heads, kv_heads) || (dim != 64 && dim != 128)) return 0;
  return woq::attn_prompt_workspace(tokens, batch, q_heads, kv_heads, dim, dtype);
}

int attn_prompt(const woq_rows *q, const woq_rows *k, const woq_rows *v, int64_t tokens, const int32_t *cu,
                int32_t batch, int32_t dim, float scale, const woq_rows *o, void *workspace,
                size_t workspace_bytes, void *stream) {
  if (!q || !k || !v || !o || !cu || tokens < 0 || batch < 1 || batch > woq::kMaxSequences) return WOQ_EINVAL;
  if (dim != 64 && dim != 128) return WOQ_ESHAPE;
  if (!prompt_heads(q->heads, k->heads)) return WOQ_EINVAL;
  const woq_rows *all[4] = {q, k, v, o};
  for (int i = 0; i < 4; ++i) {
    const int rc = woq::check_rows(all[i], tokens, i == 0 || i == 3 ? q->heads : k->heads, dim);
    if (rc != WOQ_OK) return rc;
    if (all[i]->dtype != q->dtype) return WOQ_EINVAL;
  }
  if (!woq::good_scale(scale)) return WOQ_EINVAL;
  if (!woq::aligned(cu, 4)) return WOQ_EALIGN;
  if (tokens > INT32_MAX || (tokens / 256 + batch) * q->heads > INT32_MAX) return WOQ_ESHAPE;
  const int rc_o = woq::check_written(o, tokens, dim);
  if (rc_o != WOQ_OK) return rc_o;
  if (tokens > 0)
    for (int i = 0; i < 3; ++i)
      if (woq::overlap(*all[i], *o, tokens, dim)) return WOQ_EINVAL;
  const size_t need = woq::attn_prompt_workspace(tokens, batch, q->heads, k->heads, dim, q->dtype);
  if (need > 0 && tokens > 0) {
    if (!workspace || workspace_bytes < need) return WOQ_EWORKSPACE;
    if (!woq::aligned(workspace, 256)) return WOQ_EALIGN;
  }
  DevInfo dev;
  const int rc = woq::current_device(&dev);
  if (rc != WOQ_OK || tokens == 0) return rc;
  return woq::launch_attn_prompt(*q, *k, *v, tokens, cu, batch, dim, scale, *o, workspace,
                                 static_cast<cudaStream_t>(stream), dev);
}

}  // extern "C"
