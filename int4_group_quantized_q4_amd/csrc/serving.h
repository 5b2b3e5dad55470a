// Arguments and launchers of a serving step's kernels: the plan of its rows,
// rotary positions, low-rank adapters, the draw of the next tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace w4 {

struct PlanArgs {
  const int32_t* lens;       // [seqs]; lens_out may be the same
  const int32_t* new_tokens;
  int32_t seqs;
  int32_t* table;            // [seqs][width]
  int64_t width;
  int32_t page_shift;
  int32_t* free_pages;       // [capacity]
  int64_t capacity;
  const int32_t* free_count; // free_count_out may be the same
  int32_t *lens_out, *free_count_out;
  int32_t* offsets;          // [seqs + 1]
  int64_t* slots;            // [max_rows]
  int32_t *positions, *row_seqs;   // [max_rows]; row_seqs nullable
  int64_t max_rows;
  unsigned long long* counters;    // nullable
};

void launch_plan(const PlanArgs& a, hipStream_t stream);

struct RopeArgs {
  const uint16_t *q, *k;     // k nullable with k_heads 0
  int64_t q_stride, k_stride;
  int32_t q_heads, k_heads;
  int64_t rows;
  int32_t dim, rotary;
  const int32_t* positions;
  const float* inv_freq;
  float scale;
  uint16_t *q_out, *k_out;
  int64_t q_out_stride, k_out_stride;
};

void launch_rope(const RopeArgs& a, bool interleaved, hipStream_t stream);

struct LoraArgs {
  const uint16_t* x;
  int64_t x_stride, rows;
  int32_t K;
  const int32_t* ids;
  const uint16_t *a, *b;     // [adapters][rank][K], [adapters][N][rank]
  const float* scaling;      // nullable
  int32_t adapters, rank, N;
  const uint16_t* y;
  int64_t y_stride;
  uint16_t* out;             // may be y
  int64_t out_stride;
};

size_t lora_workspace_bytes(int64_t rows, int64_t K, int64_t N, int64_t adapters, int32_t rank);
void launch_lora(const LoraArgs& a, void* ws, hipStream_t stream);

struct SampleArgs {
  const void* logits;
  int32_t dtype;             // W4_OUT_*
  int64_t rows;
  int32_t vocab;
  int64_t stride;
  const float* temperature;  // the four nullable
  const int32_t* top_k;
  const float *top_p, *min_p;
  const float* uniforms;
  int32_t* tokens;
  float* logprobs;           // nullable
};

size_t sample_workspace_bytes(int64_t rows, int64_t vocab);
void launch_sample(const SampleArgs& a, void* ws, hipStream_t stream);

}  // namespace w4
