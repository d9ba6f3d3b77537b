// Internal declarations of the 8-bit key-value cache operators (host side).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "w4a16_internal.h"

namespace w4 {
namespace kv8 {

constexpr int MAX_BATCH = 1 << 20;
constexpr int MAX_TOKENS = 1 << 24;  // new tokens of a call
constexpr int MAX_KV = 1 << 30;      // tokens that a sequence holds
constexpr int MAX_HEADS = 1024;
constexpr int MAX_DRAFTS = 64;       // of a sequence: the bits of a tree's words

// What the kernels need of a cache: pages as rows of head_dim bytes.
struct Cache {
  uint8_t *k, *v;
  float *ks, *vs;
  int pages, page_shift, heads;  // page size = 1 << page_shift
};

struct HeadRows {  // a side of the norms and rotation; heads == 0: none
  const uint16_t* in;
  uint16_t* out;
  size_t in_stride, out_stride;
  const float* weight;
  int heads;
};
struct RopeArgs {
  HeadRows rows[2];
  const float* table;
  const int32_t* positions;
  int table_rows, rot, interleaved, tokens, dim, bf16;
  float eps;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);

struct AppendArgs {
  const uint16_t *k, *v;
  size_t k_stride, v_stride;
  Cache c;
  const int32_t *table, *kv_lens, *cu_q;
  int table_stride, batch, total_q, max_q, dim, bf16;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s);

struct KeepArgs {
  Cache c;
  const int32_t *table, *kv_lens, *cu_q, *path;
  int table_stride, batch, total_q, max_q, dim;
};
cudaError_t launch_keep(const KeepArgs& a, cudaStream_t s);

struct AttnArgs {
  const uint16_t* q;
  size_t q_stride;
  Cache c;
  const int32_t *table, *kv_lens, *cu_q;
  uint16_t* out;
  int table_stride, batch, total_q, max_q, max_kv, q_heads, dim, causal, bf16;
  float scale;
  void* workspace;
  int window, sinks;     // window 0: none
  const uint64_t* tree;  // or nullptr
};
size_t attention_workspace_bytes(int batch, int max_q, int max_kv, int q_heads, int kv_heads,
                                 int dim);
cudaError_t launch_attention(const AttnArgs& a, cudaStream_t s);

struct BookArgs {
  int32_t *refs, *table, *lens;
  int pages, table_stride, seqs, page_shift;
  const int32_t *list, *list2;  // new_tokens; or drop; or src, dst; or seqs
  int n;
  int32_t *copy_src, *copy_dst;
  int32_t* status_out;
  void* workspace;
};
size_t pages_workspace_bytes(int num_pages, int n);
cudaError_t launch_reserve(const BookArgs& a, cudaStream_t s);
cudaError_t launch_fork(const BookArgs& a, cudaStream_t s);
cudaError_t launch_shorten(const BookArgs& a, cudaStream_t s);
cudaError_t launch_free(const BookArgs& a, cudaStream_t s);
cudaError_t launch_compact(const BookArgs& a, cudaStream_t s);
cudaError_t launch_copy_pages(const Cache& c, int dim, const int32_t* src, const int32_t* dst,
                              int n, cudaStream_t s);

}  // namespace kv8
}  // namespace w4
