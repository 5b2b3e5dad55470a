// extern "C" entry points of a serving step's calls (see w4a16.h): argument
// checks on the host, then kernel launches on the caller's stream.

#include <hip/hip_runtime.h>

#include "checks.h"
#include "serving.h"
#include "w4a16.h"

namespace {

struct Part {
  const void* p;
  size_t n;
};

// Whether one of the first `outputs` parts shares memory with any other part.
bool any_overlap(const Part* parts, int outputs, int count) {
  for (int i = 0; i < outputs; ++i)
    for (int j = i + 1; j < count; ++j)
      if (overlap(parts[i].p, parts[i].n, parts[j].p, parts[j].n)) return true;
  return false;
}

constexpr int64_t kMost48 = (int64_t)1 << 48;

}  // namespace

extern "C" {

int kv_cache_plan(const int32_t* seq_lens, const int32_t* new_tokens, int64_t seqs, int32_t* block_table,
                  int64_t table_width, int32_t page_size, int32_t* free_pages, int64_t capacity,
                  const int32_t* free_count, int32_t* seq_lens_out, int32_t* free_count_out, int32_t* row_offsets,
                  int64_t* slots, int32_t* positions, int32_t* row_seqs, int64_t max_rows,
                  unsigned long long* counters, hipStream_t stream) {
  if (seqs < 0 || table_width < 0 || capacity < 0 || max_rows < 0 || page_size < 1) return W4_ERR_ARG;
  if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0) return W4_ERR_SHAPE;
  if (seqs > 65535 || table_width > (int64_t)INT32_MAX / page_size || capacity > INT32_MAX ||
      max_rows > ((int64_t)1 << 26))
    return W4_ERR_SHAPE;
  if (!free_count || !free_count_out || !row_offsets || !aligned4(free_count) || !aligned4(free_count_out) ||
      !aligned4(row_offsets))
    return W4_ERR_ARG;
  if (seqs > 0 && (!seq_lens || !new_tokens || !seq_lens_out || (table_width > 0 && !block_table))) return W4_ERR_ARG;
  if (capacity > 0 && !free_pages) return W4_ERR_ARG;
  if (max_rows > 0 && (!slots || !positions)) return W4_ERR_ARG;
  if (!aligned4(seq_lens) || !aligned4(new_tokens) || !aligned4(seq_lens_out) || !aligned4(block_table) ||
      !aligned4(free_pages) || !aligned8(slots) || !aligned4(positions) || !aligned4(row_seqs) || !aligned8(counters))
    return W4_ERR_ARG;
  const size_t n = (size_t)seqs * 4;
  const Part parts[] = {{block_table, n * (size_t)table_width},
                        {free_pages, (size_t)capacity * 4},
                        {row_offsets, n + 4},
                        {slots, (size_t)max_rows * 8},
                        {positions, (size_t)max_rows * 4},
                        {row_seqs, (size_t)max_rows * 4},
                        {counters, 16},
                        {seq_lens_out, n},
                        {free_count_out, 4},
                        {new_tokens, n},
                        {seq_lens_out == seq_lens ? nullptr : seq_lens, n},
                        {free_count_out == free_count ? nullptr : free_count, 4}};
  if (any_overlap(parts, 9, 12)) return W4_ERR_ARG;
  w4::PlanArgs a{};
  a.lens = seq_lens;
  a.new_tokens = new_tokens;
  a.seqs = (int32_t)seqs;
  a.table = block_table;
  a.width = table_width;
  a.page_shift = log2_of(page_size);
  a.free_pages = free_pages;
  a.capacity = capacity;
  a.free_count = free_count;
  a.lens_out = seq_lens_out;
  a.free_count_out = free_count_out;
  a.offsets = row_offsets;
  a.slots = slots;
  a.positions = positions;
  a.row_seqs = row_seqs;
  a.max_rows = max_rows;
  a.counters = counters;
  w4::launch_plan(a, stream);
  return launch_status();
}

int w4a16_rope(const uint16_t* q, int64_t q_stride, int32_t q_heads, const uint16_t* k, int64_t k_stride,
               int32_t k_heads, int64_t rows, int32_t head_dim, int32_t rotary_dim, int32_t layout,
               const int32_t* positions, const float* inv_freq, float scale, uint16_t* q_out, int64_t q_out_stride,
               uint16_t* k_out, int64_t k_out_stride, hipStream_t stream) {
  if (rows < 0 || q_heads < 1 || k_heads < 0 || head_dim < 1 || rotary_dim < 1) return W4_ERR_ARG;
  if (layout != W4_ROPE_HALF && layout != W4_ROPE_INTERLEAVED) return W4_ERR_ARG;
  if (!(scale >= -__FLT_MAX__ && scale <= __FLT_MAX__)) return W4_ERR_ARG;
  if (head_dim % 16 != 0 || head_dim > 512 || rotary_dim % 16 != 0 || rotary_dim > head_dim) return W4_ERR_SHAPE;
  if (q_heads > 4096 || k_heads > 4096 || q_heads + k_heads > 4096 || rows >= ((int64_t)1 << 27)) return W4_ERR_SHAPE;
  if (rows == 0) return W4_OK;
  if (!positions || !inv_freq || !aligned4(positions) || !aligned4(inv_freq)) return W4_ERR_ARG;
  const int64_t qw = (int64_t)q_heads * head_dim, kw = (int64_t)k_heads * head_dim;
  int st = check_rows(q, rows, q_stride, qw);
  if (st == W4_OK) st = check_rows(q_out, rows, q_out_stride, qw);
  if (st == W4_OK && k_heads > 0) st = check_rows(k, rows, k_stride, kw);
  if (st == W4_OK && k_heads > 0) st = check_rows(k_out, rows, k_out_stride, kw);
  if (st != W4_OK) return st;
  if (k_heads == 0) k = k_out = nullptr;
  // a unit of an output is written by the thread that has read it: the same rows will do, no others
  const bool q_same = q == q_out && (q_stride == q_out_stride || rows == 1);
  const bool k_same = k == k_out && (k_stride == k_out_stride || rows == 1);
  if (!q_same && rows_overlap(q_out, q_out_stride, qw, q, q_stride, qw, rows, 2)) return W4_ERR_ARG;
  const size_t qn = rows_bytes(rows, q_out_stride, qw, 2);
  if (overlap(q_out, qn, positions, (size_t)rows * 4) || overlap(q_out, qn, inv_freq, (size_t)rotary_dim * 2))
    return W4_ERR_ARG;
  if (k) {
    if (!k_same && rows_overlap(k_out, k_out_stride, kw, k, k_stride, kw, rows, 2)) return W4_ERR_ARG;
    if (rows_overlap(q_out, q_out_stride, qw, k, k_stride, kw, rows, 2) ||
        rows_overlap(k_out, k_out_stride, kw, q, q_stride, qw, rows, 2) ||
        rows_overlap(q_out, q_out_stride, qw, k_out, k_out_stride, kw, rows, 2))
      return W4_ERR_ARG;
    const size_t kn = rows_bytes(rows, k_out_stride, kw, 2);
    if (overlap(k_out, kn, positions, (size_t)rows * 4) || overlap(k_out, kn, inv_freq, (size_t)rotary_dim * 2))
      return W4_ERR_ARG;
  }
  w4::RopeArgs a{};
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_heads = q_heads;
  a.k_heads = k_heads;
  a.rows = rows;
  a.dim = head_dim;
  a.rotary = rotary_dim;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.scale = scale;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  w4::launch_rope(a, layout == W4_ROPE_INTERLEAVED, stream);
  return launch_status();
}

static int check_lora(int64_t rows, int64_t K, int64_t N, int64_t adapters, int32_t rank) {
  if (rows < 0 || K < 0 || N < 0 || adapters < 0 || rank < 0) return W4_ERR_ARG;
  if (K < 32 || K % 32 != 0 || N % 16 != 0 || rank % 8 != 0 || rank < 8 || rank > 256) return W4_ERR_SHAPE;
  if (K > ((int64_t)1 << 20) || N > ((int64_t)1 << 20) || adapters > 4096 || rows > ((int64_t)1 << 20))
    return W4_ERR_SHAPE;
  return W4_OK;
}

size_t w4a16_lora_workspace(int64_t rows, int64_t K, int64_t N, int64_t adapters, int32_t rank) {
  if (check_lora(rows, K, N, adapters, rank) != W4_OK || rows == 0 || N == 0) return 0;
  return w4::lora_workspace_bytes(rows, K, N, adapters, rank);
}

int w4a16_lora_add(const uint16_t* x, int64_t x_stride, int64_t rows, int64_t K, const int32_t* adapter_ids,
                   const uint16_t* a, const uint16_t* b, const float* scaling, int64_t adapters, int32_t rank,
                   int64_t N, const uint16_t* y, int64_t y_stride, uint16_t* out, int64_t out_stride, void* ws,
                   size_t ws_bytes, hipStream_t stream) {
  int st = check_lora(rows, K, N, adapters, rank);
  if (st != W4_OK) return st;
  if (rows == 0 || N == 0) return W4_OK;
  if (!adapter_ids || !aligned4(adapter_ids) || !aligned4(scaling)) return W4_ERR_ARG;
  if (adapters > 0 && (!a || !b || !aligned16(a) || !aligned16(b))) return W4_ERR_ARG;
  st = check_rows(x, rows, x_stride, K);
  if (st == W4_OK) st = check_rows(y, rows, y_stride, N);
  if (st == W4_OK) st = check_rows(out, rows, out_stride, N);
  if (st != W4_OK) return st;
  const size_t need = w4a16_lora_workspace(rows, K, N, adapters, rank);
  if (need && (!ws || !aligned16(ws) || ws_bytes < need)) return W4_ERR_WORKSPACE;
  const bool same = out == y && (out_stride == y_stride || rows == 1);
  if ((!same && rows_overlap(out, out_stride, N, y, y_stride, N, rows, 2)) ||
      rows_overlap(out, out_stride, N, x, x_stride, K, rows, 2))
    return W4_ERR_ARG;
  const size_t on = rows_bytes(rows, out_stride, N, 2), an = (size_t)adapters * rank * (size_t)K * 2,
               bn = (size_t)adapters * rank * (size_t)N * 2;
  const Part parts[] = {{out, on},
                        {need ? ws : nullptr, need},
                        {adapter_ids, (size_t)rows * 4},
                        {a, an},
                        {b, bn},
                        {scaling, (size_t)adapters * 4}};
  if (any_overlap(parts, 2, 6) || overlap(ws, need, x, rows_bytes(rows, x_stride, K, 2)) ||
      overlap(ws, need, y, rows_bytes(rows, y_stride, N, 2)))
    return W4_ERR_ARG;
  w4::LoraArgs l{};
  l.x = x;
  l.x_stride = x_stride;
  l.rows = rows;
  l.K = (int32_t)K;
  l.ids = adapter_ids;
  l.a = a;
  l.b = b;
  l.scaling = scaling;
  l.adapters = (int32_t)adapters;
  l.rank = rank;
  l.N = (int32_t)N;
  l.y = y;
  l.y_stride = y_stride;
  l.out = out;
  l.out_stride = out_stride;
  w4::launch_lora(l, ws, stream);
  return launch_status();
}

static int check_sample(int64_t rows, int64_t vocab) {
  if (rows < 0 || vocab < 0) return W4_ERR_ARG;
  if (vocab < 1 || vocab > ((int64_t)1 << 20) || rows > 65535) return W4_ERR_SHAPE;
  return W4_OK;
}

size_t w4a16_sample_workspace(int64_t rows, int64_t vocab) {
  if (check_sample(rows, vocab) != W4_OK || rows == 0) return 0;
  return w4::sample_workspace_bytes(rows, vocab);
}

int w4a16_sample(const void* logits, int32_t logits_dtype, int64_t rows, int64_t vocab, int64_t stride,
                 const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                 const float* uniforms, int32_t* tokens, float* logprobs, void* ws, size_t ws_bytes,
                 hipStream_t stream) {
  if (logits_dtype != W4_OUT_BF16 && logits_dtype != W4_OUT_F32) return W4_ERR_ARG;
  const int st = check_sample(rows, vocab);
  if (st != W4_OK) return st;
  if (rows == 0) return W4_OK;
  const int64_t element = logits_dtype == W4_OUT_F32 ? 4 : 2;
  if (!logits || (reinterpret_cast<uintptr_t>(logits) & (uintptr_t)(element - 1)) || stride < vocab) return W4_ERR_ARG;
  if (stride > kMost48 / rows) return W4_ERR_SHAPE;
  if (!uniforms || !tokens || !aligned4(uniforms) || !aligned4(tokens) || !aligned4(logprobs) ||
      !aligned4(temperature) || !aligned4(top_k) || !aligned4(top_p) || !aligned4(min_p))
    return W4_ERR_ARG;
  const size_t need = w4a16_sample_workspace(rows, vocab);
  if (need && (!ws || !aligned16(ws) || ws_bytes < need)) return W4_ERR_WORKSPACE;
  const size_t n = (size_t)rows * 4;
  const Part parts[] = {{tokens, n},      {logprobs, n}, {need ? ws : nullptr, need},
                        {temperature, n}, {top_k, n},    {top_p, n},
                        {min_p, n},       {uniforms, n}, {logits, rows_bytes(rows, stride, vocab, element)}};
  if (any_overlap(parts, 3, 9)) return W4_ERR_ARG;
  w4::SampleArgs a{};
  a.logits = logits;
  a.dtype = logits_dtype;
  a.rows = rows;
  a.vocab = (int32_t)vocab;
  a.stride = stride;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.uniforms = uniforms;
  a.tokens = tokens;
  a.logprobs = logprobs;
  w4::launch_sample(a, ws, stream);
  return launch_status();
}

}  // extern "C"
