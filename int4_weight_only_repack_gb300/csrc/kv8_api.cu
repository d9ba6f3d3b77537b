// C ABI of the 8-bit key-value cache (the w4_kv8_* entry points of
// include/w4a16.h, and w4_qk_norm_rope before them): argument validation and dispatch. Every check runs on the
// host before any CUDA call; nothing is launched on error. Table entries,
// lengths and offsets live on the device and are checked by the kernels.
#include <cuda_runtime.h>

#include <cmath>

#include "kv8_internal.h"

using namespace w4;
using namespace w4::kv8;

namespace {

constexpr int MAX_PAGES = 1 << 26;

w4_status check_page_size(int page_size) {
  return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 ? W4_OK
                                                                                   : W4_ERR_SHAPE;
}

int shift_of(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

w4_status check_cache(const w4_kv8_cache* c) {
  if (!c) return W4_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128) return W4_ERR_SHAPE;
  if (check_page_size(c->page_size) || c->kv_heads < 1 || c->kv_heads > MAX_HEADS ||
      c->num_pages < 1 || c->num_pages > MAX_PAGES)
    return W4_ERR_SHAPE;
  // token rows are addressed with 32-bit coordinates (2^31 rows of 128 bytes are 256 GiB)
  if ((long long)c->num_pages * c->kv_heads * c->page_size >= (1ll << 31)) return W4_ERR_SHAPE;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return W4_ERR_NULL;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
    return W4_ERR_ALIGN;
  return W4_OK;
}

size_t code_bytes(const w4_kv8_cache* c) {
  return (size_t)c->num_pages * c->kv_heads * c->page_size * c->head_dim;
}
size_t scale_bytes(const w4_kv8_cache* c) { return (size_t)c->num_pages * c->kv_heads * 4; }

// Whether a buffer overlaps one of the cache's four.
bool overlaps_cache(const w4_kv8_cache* c, const void* p, size_t n) {
  return overlaps(p, n, c->k, code_bytes(c)) || overlaps(p, n, c->v, code_bytes(c)) ||
         overlaps(p, n, c->k_scale, scale_bytes(c)) || overlaps(p, n, c->v_scale, scale_bytes(c));
}

bool cache_overlaps_itself(const w4_kv8_cache* c) {
  const size_t cb = code_bytes(c), sb = scale_bytes(c);
  return overlaps(c->k, cb, c->v, cb) || overlaps(c->k, cb, c->k_scale, sb) ||
         overlaps(c->k, cb, c->v_scale, sb) || overlaps(c->v, cb, c->k_scale, sb) ||
         overlaps(c->v, cb, c->v_scale, sb) || overlaps(c->k_scale, sb, c->v_scale, sb);
}

Cache device_cache(const w4_kv8_cache* c) {
  return {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scale, c->v_scale,
          c->num_pages, shift_of(c->page_size), c->kv_heads};
}

// The integer arrays may be slices of larger ones: int32 alignment is enough.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The arguments append and attention share.
w4_status check_batch(const int32_t* table, int table_stride, const int32_t* kv_lens,
                      const int32_t* cu_q, int batch, int total_q, int max_q_len, int dtype) {
  if (dtype != W4_F16 && dtype != W4_BF16) return W4_ERR_DTYPE;
  if (batch < 0 || batch > MAX_BATCH || total_q < 0 || total_q > MAX_TOKENS || max_q_len < 0 ||
      max_q_len > MAX_TOKENS || table_stride < 1)
    return W4_ERR_SHAPE;
  if (batch > 0 && (!table || !kv_lens || !cu_q)) return W4_ERR_NULL;
  if (!aligned4(table) || !aligned4(kv_lens) || !aligned4(cu_q)) return W4_ERR_ALIGN;
  return W4_OK;
}

size_t table_bytes(int rows, int stride) { return (size_t)rows * stride * 4; }

// Extent in bytes of `rows` 16-bit rows of `width` elements, `stride` apart.
size_t strided_bytes(int rows, size_t stride, int width) {
  return rows > 0 ? ((size_t)(rows - 1) * stride + width) * 2 : 0;
}
// Rows begin on 16-byte boundaries and do not overlap.
bool bad_stride(size_t stride, int width) {
  return stride < (size_t)width || stride % 8 || stride > ((size_t)1 << 40);
}

w4_status check_pool(const int32_t* refs, int num_pages, const int32_t* table, int table_stride,
                     int num_seqs) {
  if (num_pages < 1 || num_pages > MAX_PAGES || table_stride < 1 || num_seqs < 0 ||
      num_seqs > MAX_BATCH)
    return W4_ERR_SHAPE;
  if (!refs || (num_seqs > 0 && !table)) return W4_ERR_NULL;
  if (!aligned4(refs) || !aligned4(table)) return W4_ERR_ALIGN;
  return W4_OK;
}

// Integer buffers that a call writes (the first `writes` of them) must not
// overlap one another or the ones it reads.
struct Extent {
  const void* p;
  size_t n;
};
bool any_alias(const Extent* e, int count, int writes) {
  for (int i = 0; i < writes; ++i)
    for (int j = i + 1; j < count; ++j)
      if (overlaps(e[i].p, e[i].n, e[j].p, e[j].n)) return true;
  return false;
}

// Whether two sides' rows share bytes: `tokens` rows of wa and wb bytes, sa and sb bytes
// apart. Rows of one buffer (slices of a projection) lie at one stride and differ in
// where they begin within it.
bool rows_overlap(const void* a, size_t sa, size_t wa, const void* b, size_t sb, size_t wb, int tokens) {
  const size_t last = (size_t)(tokens - 1);
  if (!overlaps(a, last * sa + wa, b, last * sb + wb)) return false;
  if (sa != sb) return true;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const size_t d = b0 >= a0 ? (b0 - a0) % sa : (sa - (a0 - b0) % sa) % sa;
  return d < wa || d + wb > sa;
}

w4_status check_side(const w4_head_rows* r, int head_dim) {
  if (r->heads < 1 || r->heads > MAX_HEADS || bad_stride(r->in_stride, r->heads * head_dim) ||
      bad_stride(r->out_stride, r->heads * head_dim))
    return W4_ERR_SHAPE;
  if (!r->in || !r->out) return W4_ERR_NULL;
  if (!aligned16(r->in) || !aligned16(r->out) || !aligned16(r->weight)) return W4_ERR_ALIGN;
  return W4_OK;
}

// Both attention calls.
w4_status attend(const void* q, size_t q_stride, const w4_kv8_cache* cache, const int32_t* table,
                 int table_stride, const int32_t* kv_lens, const int32_t* cu_q, void* out, int batch,
                 int total_q, int max_q_len, int max_kv_len, const w4_kv8_heads* heads,
                 const w4_kv8_mask& mask, int dtype, void* workspace, size_t workspace_bytes,
                 void* stream) {
  w4_status st = check_cache(cache);
  if (st) return st;
  if (!heads) return W4_ERR_NULL;
  const int q_heads = heads->q_heads;
  if ((st = check_batch(table, table_stride, kv_lens, cu_q, batch, total_q, max_q_len, dtype)))
    return st;
  if (q_heads < 1 || q_heads > MAX_HEADS || q_heads % cache->kv_heads || max_kv_len < 0 ||
      max_kv_len > MAX_KV || heads->causal < 0 || heads->causal > 1 || !std::isfinite(heads->scale))
    return W4_ERR_SHAPE;
  const int width = q_heads * cache->head_dim;
  if (bad_stride(q_stride, width)) return W4_ERR_SHAPE;
  if (batch == 0 || total_q == 0 || max_q_len == 0) return W4_OK;
  if (!q || !out) return W4_ERR_NULL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return W4_ERR_ALIGN;
  const size_t need = w4_kv8_attention_workspace_size(batch, total_q, max_q_len, max_kv_len,
                                                      q_heads, cache->kv_heads, cache->head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return W4_ERR_WORKSPACE;
  const size_t out_b = strided_bytes(total_q, width, width);
  const Extent e[7] = {{out, out_b},
                       {workspace, workspace ? need : 0},
                       {q, strided_bytes(total_q, q_stride, width)},
                       {table, table_bytes(batch, table_stride)},
                       {kv_lens, (size_t)batch * 4},
                       {cu_q, (size_t)(batch + 1) * 4},
                       {mask.tree, (size_t)total_q * 8}};
  if (any_alias(e, 7, 2) || overlaps_cache(cache, out, out_b) ||
      overlaps_cache(cache, workspace, workspace ? need : 0))
    return W4_ERR_ALIAS;
  if ((st = check_arch())) return st;
  AttnArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.c = device_cache(cache);
  a.table = table;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.out = static_cast<uint16_t*>(out);
  a.table_stride = table_stride;
  a.batch = batch;
  a.total_q = total_q;
  a.max_q = max_q_len;
  a.max_kv = max_kv_len;
  a.q_heads = q_heads;
  a.dim = cache->head_dim;
  a.causal = heads->causal;
  a.bf16 = dtype == W4_BF16;
  a.scale = heads->scale;
  a.workspace = workspace;
  a.window = mask.window;
  a.sinks = mask.sinks;
  a.tree = mask.tree;
  const std::lock_guard<std::mutex> lock(stream_mutex(stream));
  return from_cuda(launch_attention(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

w4_status w4_qk_norm_rope(const w4_head_rows* q, const w4_head_rows* k, const w4_norm_rope* how,
                          const int32_t* positions, int tokens, int head_dim, int dtype, void* stream) {
  if (dtype != W4_F16 && dtype != W4_BF16) return W4_ERR_DTYPE;
  if (!how) return W4_ERR_NULL;
  if ((head_dim != 64 && head_dim != 128) || tokens < 0 || tokens > MAX_TOKENS || !(how->eps >= 0.f) ||
      !std::isfinite(how->eps))
    return W4_ERR_SHAPE;
  const w4_head_rows* sides[2] = {q, k};
  const bool turns = how->table != nullptr;
  bool does = turns;
  for (const w4_head_rows* s : sides) does = does || (s && s->weight);
  if ((!q && !k) || !does) return W4_ERR_NULL;
  if (turns && (how->rows < 1 || how->rot_dim < 16 || how->rot_dim > head_dim || how->rot_dim % 16 ||
                how->interleaved < 0 || how->interleaved > 1))
    return W4_ERR_SHAPE;
  if (tokens == 0) return W4_OK;
  w4_status st;
  for (const w4_head_rows* s : sides)
    if (s && (st = check_side(s, head_dim))) return st;
  if (turns && !positions) return W4_ERR_NULL;
  if (!aligned16(how->table) || !aligned4(positions)) return W4_ERR_ALIGN;
  // an output shares no byte with anything else, but for its own input in place
  const size_t table_b = turns ? (size_t)how->rows * how->rot_dim * 4 : 0;
  for (const w4_head_rows* s : sides) {
    if (!s) continue;
    const size_t stride = s->out_stride * 2, width = (size_t)s->heads * head_dim * 2;
    const size_t all = (size_t)(tokens - 1) * stride + width;
    if (overlaps(s->out, all, how->table, table_b) || overlaps(s->out, all, positions, (size_t)tokens * 4))
      return W4_ERR_ALIAS;
    for (const w4_head_rows* o : sides) {
      if (!o) continue;
      const size_t wide = (size_t)o->heads * head_dim * 2;
      if (overlaps(s->out, all, o->weight, (size_t)head_dim * 4)) return W4_ERR_ALIAS;
      const bool in_place = o == s && s->out == s->in && s->out_stride == s->in_stride;
      if (!in_place && rows_overlap(s->out, stride, width, o->in, o->in_stride * 2, wide, tokens)) return W4_ERR_ALIAS;
      if (o != s && rows_overlap(s->out, stride, width, o->out, o->out_stride * 2, wide, tokens)) return W4_ERR_ALIAS;
    }
  }
  if ((st = check_arch())) return st;
  RopeArgs a = {};
  for (int i = 0; i < 2; ++i)
    if (const w4_head_rows* s = sides[i])
      a.rows[i] = {static_cast<const uint16_t*>(s->in), static_cast<uint16_t*>(s->out), s->in_stride,
                   s->out_stride, s->weight, s->heads};
  if (turns) {
    a.table = how->table;
    a.table_rows = how->rows;
    a.rot = how->rot_dim;
    a.interleaved = how->interleaved;
  }
  a.positions = positions;
  a.tokens = tokens;
  a.dim = head_dim;
  a.bf16 = dtype == W4_BF16;
  a.eps = how->eps;
  return from_cuda(launch_rope(a, static_cast<cudaStream_t>(stream)));
}

w4_status w4_kv8_append(const void* k_new, const void* v_new, size_t k_stride, size_t v_stride,
                        const w4_kv8_cache* cache, const int32_t* table,
                        int table_stride, const int32_t* kv_lens, const int32_t* cu_q, int batch,
                        int total_q, int max_q_len, int dtype, void* stream) {
  w4_status st = check_cache(cache);
  if (st) return st;
  if ((st = check_batch(table, table_stride, kv_lens, cu_q, batch, total_q, max_q_len, dtype)))
    return st;
  const int width = cache->kv_heads * cache->head_dim;
  if (bad_stride(k_stride, width) || bad_stride(v_stride, width)) return W4_ERR_SHAPE;
  if (batch == 0 || total_q == 0 || max_q_len == 0) return W4_OK;
  if (!k_new || !v_new) return W4_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new)) return W4_ERR_ALIGN;
  if (overlaps_cache(cache, k_new, strided_bytes(total_q, k_stride, width)) ||
      overlaps_cache(cache, v_new, strided_bytes(total_q, v_stride, width)) ||
      overlaps_cache(cache, table, table_bytes(batch, table_stride)) ||
      overlaps_cache(cache, kv_lens, (size_t)batch * 4) ||
      overlaps_cache(cache, cu_q, (size_t)(batch + 1) * 4) || cache_overlaps_itself(cache))
    return W4_ERR_ALIAS;
  if ((st = check_arch())) return st;
  AppendArgs a;
  a.k = static_cast<const uint16_t*>(k_new);
  a.v = static_cast<const uint16_t*>(v_new);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.c = device_cache(cache);
  a.table = table;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.table_stride = table_stride;
  a.batch = batch;
  a.total_q = total_q;
  a.max_q = max_q_len;
  a.dim = cache->head_dim;
  a.bf16 = dtype == W4_BF16;
  return from_cuda(launch_append(a, static_cast<cudaStream_t>(stream)));
}

size_t w4_kv8_attention_workspace_size(int batch, int total_q, int max_q_len, int max_kv_len,
                                       int q_heads, int kv_heads, int head_dim) {
  if (batch < 1 || batch > MAX_BATCH || total_q < 1 || total_q > MAX_TOKENS || max_q_len < 1 ||
      max_q_len > MAX_TOKENS || max_kv_len < 0 || max_kv_len > MAX_KV || q_heads < 1 ||
      q_heads > MAX_HEADS || kv_heads < 1 || q_heads % kv_heads || (head_dim != 64 && head_dim != 128))
    return 0;
  return attention_workspace_bytes(batch, max_q_len, max_kv_len, q_heads, kv_heads, head_dim);
}

w4_status w4_kv8_attention(const void* q, size_t q_stride, const w4_kv8_cache* cache,
                           const int32_t* table, int table_stride, const int32_t* kv_lens,
                           const int32_t* cu_q, void* out, int batch, int total_q, int max_q_len,
                           int max_kv_len, const w4_kv8_heads* heads, int dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const w4_kv8_mask none = {0, 0, nullptr};
  return attend(q, q_stride, cache, table, table_stride, kv_lens, cu_q, out, batch, total_q, max_q_len,
                max_kv_len, heads, none, dtype, workspace, workspace_bytes, stream);
}

w4_status w4_kv8_attention_masked(const void* q, size_t q_stride, const w4_kv8_cache* cache,
                                  const int32_t* table, int table_stride, const int32_t* kv_lens,
                                  const int32_t* cu_q, void* out, int batch, int total_q,
                                  int max_q_len, int max_kv_len, const w4_kv8_heads* heads,
                                  const w4_kv8_mask* mask, int dtype, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!mask || (mask->window == 0 && !mask->tree)) return W4_ERR_NULL;
  if (mask->window < 0 || mask->sinks < 0 || mask->sinks > MAX_KV || (mask->sinks > 0 && mask->window == 0) ||
      (heads && heads->causal != 1) || (mask->tree && max_q_len > MAX_DRAFTS))
    return W4_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(mask->tree) & 7u) return W4_ERR_ALIGN;
  return attend(q, q_stride, cache, table, table_stride, kv_lens, cu_q, out, batch, total_q, max_q_len,
                max_kv_len, heads, *mask, dtype, workspace, workspace_bytes, stream);
}

w4_status w4_kv8_keep(const w4_kv8_cache* cache, const int32_t* table, int table_stride,
                      const int32_t* kv_lens, const int32_t* cu_q, const int32_t* path, int batch,
                      int total_q, int max_q_len, void* stream) {
  w4_status st = check_cache(cache);
  if (st) return st;
  if ((st = check_batch(table, table_stride, kv_lens, cu_q, batch, total_q, max_q_len, W4_F16))) return st;
  if (max_q_len > MAX_DRAFTS) return W4_ERR_SHAPE;
  if (batch == 0 || total_q == 0 || max_q_len == 0) return W4_OK;
  if (!path) return W4_ERR_NULL;
  if (!aligned4(path)) return W4_ERR_ALIGN;
  if (overlaps_cache(cache, table, table_bytes(batch, table_stride)) ||
      overlaps_cache(cache, kv_lens, (size_t)batch * 4) || overlaps_cache(cache, cu_q, (size_t)(batch + 1) * 4) ||
      overlaps_cache(cache, path, (size_t)total_q * 4) || cache_overlaps_itself(cache))
    return W4_ERR_ALIAS;
  if ((st = check_arch())) return st;
  const KeepArgs a{device_cache(cache), table, kv_lens, cu_q, path, table_stride, batch, total_q, max_q_len,
                   cache->head_dim};
  return from_cuda(launch_keep(a, static_cast<cudaStream_t>(stream)));
}

size_t w4_kv8_pages_workspace_size(int num_pages, int n) {
  if (num_pages < 1 || num_pages > MAX_PAGES || n < 0 || n > MAX_BATCH) return 0;
  return pages_workspace_bytes(num_pages, n);
}

w4_status w4_kv8_reserve(int32_t* refs, int num_pages, int32_t* table, int table_stride,
                         int32_t* lens, int num_seqs, const int32_t* new_tokens, int page_size,
                         int32_t* status_out, void* workspace, size_t workspace_bytes,
                         void* stream) {
  w4_status st = check_pool(refs, num_pages, table, table_stride, num_seqs);
  if (st) return st;
  if ((st = check_page_size(page_size))) return st;
  if (num_seqs > 0 && (!lens || !new_tokens)) return W4_ERR_NULL;
  if (!aligned4(lens) || !aligned4(new_tokens) || !aligned4(status_out) || !aligned16(workspace))
    return W4_ERR_ALIGN;
  const size_t need = pages_workspace_bytes(num_pages, num_seqs);
  if (!workspace || workspace_bytes < need) return W4_ERR_WORKSPACE;
  const size_t s4 = (size_t)num_seqs * 4;
  const Extent e[6] = {{refs, (size_t)num_pages * 4}, {table, table_bytes(num_seqs, table_stride)},
                       {lens, s4}, {workspace, need}, {status_out, status_out ? 4u : 0u},
                       {new_tokens, s4}};
  if (any_alias(e, 6, 5)) return W4_ERR_ALIAS;
  if ((st = check_arch())) return st;
  BookArgs a{refs, table, lens, num_pages, table_stride, num_seqs, shift_of(page_size), new_tokens,
             nullptr, num_seqs, nullptr, nullptr, status_out, workspace};
  return from_cuda(launch_reserve(a, static_cast<cudaStream_t>(stream)));
}

w4_status w4_kv8_shorten(int32_t* refs, int num_pages, int32_t* table, int table_stride,
                         int32_t* lens, int num_seqs, const int32_t* drop, int page_size,
                         int32_t* status_out, void* stream) {
  w4_status st = check_pool(refs, num_pages, table, table_stride, num_seqs);
  if (st) return st;
  if ((st = check_page_size(page_size))) return st;
  if (num_seqs > 0 && (!lens || !drop)) return W4_ERR_NULL;
  if (!aligned4(lens) || !aligned4(drop) || !aligned4(status_out)) return W4_ERR_ALIGN;
  const size_t s4 = (size_t)num_seqs * 4;
  const Extent e[5] = {{refs, (size_t)num_pages * 4}, {table, table_bytes(num_seqs, table_stride)}, {lens, s4},
                       {status_out, status_out ? 4u : 0u}, {drop, s4}};
  if (any_alias(e, 5, 4)) return W4_ERR_ALIAS;
  if ((st = check_arch())) return st;
  BookArgs a{refs, table, lens, num_pages, table_stride, num_seqs, shift_of(page_size), drop, nullptr,
             num_seqs, nullptr, nullptr, status_out, nullptr};
  return from_cuda(launch_shorten(a, static_cast<cudaStream_t>(stream)));
}

w4_status w4_kv8_fork(int32_t* refs, int num_pages, int32_t* table, int table_stride,
                      int32_t* lens, int num_seqs, const int32_t* src, const int32_t* dst, int n,
                      int page_size, int32_t* copy_src, int32_t* copy_dst, int32_t* status_out,
                      void* workspace, size_t workspace_bytes, void* stream) {
  w4_status st = check_pool(refs, num_pages, table, table_stride, num_seqs);
  if (st) return st;
  if ((st = check_page_size(page_size))) return st;
  if (n < 0 || n > num_seqs) return W4_ERR_SHAPE;
  if (num_seqs > 0 && !lens) return W4_ERR_NULL;
  if (n > 0 && (!src || !dst || !copy_src || !copy_dst)) return W4_ERR_NULL;
  if (!aligned4(lens) || !aligned4(src) || !aligned4(dst) || !aligned4(copy_src) ||
      !aligned4(copy_dst) || !aligned4(status_out) || !aligned16(workspace))
    return W4_ERR_ALIGN;
  const size_t need = pages_workspace_bytes(num_pages, n);
  if (!workspace || workspace_bytes < need) return W4_ERR_WORKSPACE;
  const size_t n4 = (size_t)n * 4;
  const Extent e[9] = {{refs, (size_t)num_pages * 4}, {table, table_bytes(num_seqs, table_stride)},
                       {lens, (size_t)num_seqs * 4}, {workspace, need}, {copy_src, n4},
                       {copy_dst, n4}, {status_out, status_out ? 4u : 0u}, {src, n4}, {dst, n4}};
  if (any_alias(e, 9, 7)) return W4_ERR_ALIAS;
  if ((st = check_arch())) return st;
  BookArgs a{refs, table, lens, num_pages, table_stride, num_seqs, shift_of(page_size), src, dst, n,
             copy_src, copy_dst, status_out, workspace};
  return from_cuda(launch_fork(a, static_cast<cudaStream_t>(stream)));
}

w4_status w4_kv8_free(int32_t* refs, int num_pages, int32_t* table, int table_stride,
                      int32_t* lens, int num_seqs, const int32_t* seqs, int n, int page_size,
                      int32_t* status_out, void* stream) {
  w4_status st = check_pool(refs, num_pages, table, table_stride, num_seqs);
  if (st) return st;
  if ((st = check_page_size(page_size))) return st;
  if (n < 0 || n > MAX_BATCH) return W4_ERR_SHAPE;
  if ((num_seqs > 0 && !lens) || (n > 0 && !seqs)) return W4_ERR_NULL;
  if (!aligned4(lens) || !aligned4(seqs) || !aligned4(status_out)) return W4_ERR_ALIGN;
  const Extent e[5] = {{refs, (size_t)num_pages * 4}, {table, table_bytes(num_seqs, table_stride)},
                       {lens, (size_t)num_seqs * 4}, {status_out, status_out ? 4u : 0u},
                       {seqs, (size_t)n * 4}};
  if (any_alias(e, 5, 4)) return W4_ERR_ALIAS;
  if ((st = check_arch())) return st;
  BookArgs a{refs, table, lens, num_pages, table_stride, num_seqs, shift_of(page_size), seqs,
             nullptr, n, nullptr, nullptr, status_out, nullptr};
  const std::lock_guard<std::mutex> lock(stream_mutex(stream));
  return from_cuda(launch_free(a, static_cast<cudaStream_t>(stream)));
}

w4_status w4_kv8_compact(int32_t* refs, int num_pages, int32_t* table, int table_stride,
                         int num_seqs, int32_t* copy_src, int32_t* copy_dst, void* workspace,
                         size_t workspace_bytes, void* stream) {
  w4_status st = check_pool(refs, num_pages, table, table_stride, num_seqs);
  if (st) return st;
  if (!copy_src || !copy_dst) return W4_ERR_NULL;
  if (!aligned4(copy_src) || !aligned4(copy_dst) || !aligned16(workspace)) return W4_ERR_ALIGN;
  const size_t need = pages_workspace_bytes(num_pages, num_seqs);
  if (!workspace || workspace_bytes < need) return W4_ERR_WORKSPACE;
  const size_t p4 = (size_t)num_pages * 4;
  const Extent e[5] = {{refs, p4}, {table, table_bytes(num_seqs, table_stride)}, {workspace, need},
                       {copy_src, p4}, {copy_dst, p4}};
  if (any_alias(e, 5, 5)) return W4_ERR_ALIAS;
  if ((st = check_arch())) return st;
  BookArgs a{refs, table, nullptr, num_pages, table_stride, num_seqs, 0, nullptr, nullptr, 0,
             copy_src, copy_dst, nullptr, workspace};
  const std::lock_guard<std::mutex> lock(stream_mutex(stream));
  return from_cuda(launch_compact(a, static_cast<cudaStream_t>(stream)));
}

w4_status w4_kv8_copy_pages(const w4_kv8_cache* cache, const int32_t* src, const int32_t* dst,
                            int n, void* stream) {
  w4_status st = check_cache(cache);
  if (st) return st;
  if (n < 0 || n > MAX_PAGES) return W4_ERR_SHAPE;
  if (n == 0) return W4_OK;
  if (!src || !dst) return W4_ERR_NULL;
  if (!aligned4(src) || !aligned4(dst)) return W4_ERR_ALIGN;
  if (overlaps_cache(cache, src, (size_t)n * 4) || overlaps_cache(cache, dst, (size_t)n * 4) ||
      cache_overlaps_itself(cache))
    return W4_ERR_ALIAS;
  if ((st = check_arch())) return st;
  return from_cuda(launch_copy_pages(device_cache(cache), cache->head_dim, src, dst, n,
                                     static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
