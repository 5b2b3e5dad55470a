// Arguments and launchers of the norm, key-value cache and attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace w4 {

// y (bf16) or q and scale (E4M3), the other null; residual and sum_out nullable
void launch_add_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t rows, int64_t d,
                        float eps, float offset, uint16_t* sum_out, uint16_t* y, uint8_t* q, float* scale,
                        hipStream_t stream);

// Rows written into the key-value cache or read back from it.
struct KvArgs {
  int32_t format;            // W4_KV_*
  uint8_t* cache;
  int64_t n_pages;
  int32_t page_shift;        // log2 of the tokens per page
  int32_t kv_heads, head_dim;
  int64_t block_bytes;       // of one head's K (or V) rows in a page
  int64_t page_bytes;        // kv_heads * 2 * block_bytes
  const int64_t* slots;      // [tokens]
  int64_t tokens;
  const uint16_t *k, *v;     // write: rows of kv_heads * head_dim bf16, strides in elements
  void *k_out, *v_out;       // read
  int64_t k_stride, v_stride;
  unsigned long long* counters;   // nullable
};

void launch_kv_write(const KvArgs& a, hipStream_t stream);
void launch_kv_read(const KvArgs& a, int out_dtype, hipStream_t stream);

// One-token attention over the paged cache.
struct AttnArgs {
  const uint16_t* q;         // [seqs] rows of heads * head_dim bf16, q_stride elements apart
  int64_t seqs, q_stride;
  int32_t heads;
  int32_t format;
  const uint8_t* cache;
  int64_t n_pages;
  int32_t page_shift, kv_heads, head_dim;
  int64_t block_bytes, page_bytes;
  const int32_t* table;      // [seqs][table_width]
  int64_t table_width;
  const int32_t* lens;       // [seqs]
  float scale;
  int32_t window;
  uint16_t* out;             // [seqs][heads][head_dim]
  float* lse;                // nullable, [seqs][heads]
  unsigned long long* counters;   // nullable
  // set by launch_kv_attention
  int32_t head_tiles;
  int32_t shares;            // equal shares that the positions are cut into; 0: no splits
  float* part_o;             // [items][heads][head_dim]
  float* part_ml;            // [items][heads][2]
  int2* part_plan;           // [seqs]: first item, items
};

size_t kv_attention_workspace_bytes(int64_t seqs, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t tokens);
void launch_kv_attention(AttnArgs a, void* ws, hipStream_t stream);

}  // namespace w4
