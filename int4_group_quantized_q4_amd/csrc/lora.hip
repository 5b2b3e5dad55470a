// Low-rank adapters of many requests beside a projection:
//   out[t] = bf16(y[t] + s_i (x[t] A_i^T) B_i^T),  i = ids[t].

#include "common.h"
#include "serving.h"

namespace w4 {

namespace {

constexpr int kLoraThreads = 256;

// h[t][r] = s_i sum_k x[t][k] a[i][r][k]: a wave per r
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_kernel(LoraArgs l, float* h) {
  const int64_t t = blockIdx.x;
  const int id = l.ids[t], lane = threadIdx.x & 63;
  if (id < 0 || id >= l.adapters) return;
  const u32x4* xs = reinterpret_cast<const u32x4*>(l.x + t * l.x_stride);
  const float s = l.scaling ? l.scaling[id] : 1.0f;
  for (int r = threadIdx.x >> 6; r < l.rank; r += kLoraThreads / 64) {
    const u32x4* as = reinterpret_cast<const u32x4*>(l.a + ((int64_t)id * l.rank + r) * l.K);
    float sum = 0.f;
    for (int c = lane; c < l.K / 8; c += 64) {
      const u32x4 v = xs[c], w = as[c];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum = __builtin_fmaf(bf16_to_f32(v[j] & 0xFFFFu), bf16_to_f32(w[j] & 0xFFFFu), sum);
        sum = __builtin_fmaf(__uint_as_float(v[j] & 0xFFFF0000u), __uint_as_float(w[j] & 0xFFFF0000u), sum);
      }
    }
    sum = wave_sum_all(sum);
    if (lane == 0) h[t * l.rank + r] = sum * s;
  }
}

__global__ void __launch_bounds__(kLoraThreads) lora_expand_kernel(LoraArgs l, const float* h) {
  const int64_t t = blockIdx.x;
  const int n = blockIdx.y * kLoraThreads + threadIdx.x;
  if (n >= l.N) return;
  const int id = l.ids[t];
  uint16_t* to = l.out + t * l.out_stride + n;
  const uint16_t old = l.y[t * l.y_stride + n];
  if (id < 0 || id >= l.adapters) {
    *to = old;
    return;
  }
  const uint16_t* bs = l.b + ((int64_t)id * l.N + n) * l.rank;
  float sum = 0.f;
  for (int r = 0; r < l.rank; ++r) sum = __builtin_fmaf(h[t * l.rank + r], bf16_to_f32(bs[r]), sum);
  *to = bf16_rne(bf16_to_f32(old) + sum);
}

}  // namespace

size_t lora_workspace_bytes(int64_t rows, int64_t, int64_t, int64_t, int32_t rank) {
  return (size_t)rows * (size_t)rank * sizeof(float);
}

void launch_lora(const LoraArgs& l, void* ws, hipStream_t stream) {
  float* h = static_cast<float*>(ws);
  // a launch holds fewer than 2^32 threads
  constexpr int64_t kSlice = (int64_t)1 << 16;
  for (int64_t r0 = 0; r0 < l.rows; r0 += kSlice) {
    LoraArgs s = l;
    s.rows = l.rows - r0 < kSlice ? l.rows - r0 : kSlice;
    s.x += r0 * l.x_stride;
    s.ids += r0;
    s.y += r0 * l.y_stride;
    s.out += r0 * l.out_stride;
    lora_shrink_kernel<<<(unsigned)s.rows, kLoraThreads, 0, stream>>>(s, h + r0 * l.rank);
    lora_expand_kernel<<<dim3((unsigned)s.rows, (unsigned)((l.N + kLoraThreads - 1) / kLoraThreads)), kLoraThreads, 0,
                         stream>>>(s, h + r0 * l.rank);
  }
}

}  // namespace w4
