// Rotary positions of queries and keys.
//
//   (a, b) -> scale (a cos t - b sin t, b cos t + a sin t),  t = p f_j
//
// The angle is taken in turns: u = t / (2 pi) as two 64-bit terms (the product of
// a 31-bit position and a 24-bit frequency, which has 55 bits and so two terms of
// its own, times 1 / (2 pi) to 106 bits), less the nearest quarter turn, exactly,
// so that the fp32 sine and cosine are of an angle within an eighth of a turn that
// is good to its last bit, and the quarters swap and negate them.  (In fp32, as the
// turned elements keep 8 bits: their error is 2^-15 of that rounding.)
//
// Bound by memory for many rows: every element is read and written once (8191 rows
// of 20 heads of 256, half of each turned: 34.3 us, 4.9 TB/s, where a call's rows come
// from memory; 26.7 where it is repeated on the same 168 MB, half of whose reads the
// last-level cache then answers), by latency for few (a row of 40 heads of 128 2.7 us,
// 64 rows 3.4).  The angles of a row are common to its
// heads: a workgroup takes whole rows (or a part of one) and computes each angle once,
// into LDS.

#include "common.h"
#include "serving.h"

namespace w4 {

namespace {

constexpr int kRopeThreads = 256;
// Units, 16 dimensions of a head each, of one thread: two share an angle's cost (8191
// rows as above, repeated, 26.7 us, 32.7 with one, 27.5 with four), one where that leaves
// CUs without work (64 rows 3.5 against 3.9 us in a graph).
constexpr int kFewUnits = 256 * kRopeThreads * 2;

struct RopeTile {
  int32_t units, q_units;      // units in a row, and in its queries
  int32_t head_units, turned;  // units in a head, and those of its turned dimensions
  int32_t rows;                // rows a workgroup takes
  int32_t parts;               // workgroups a row takes (rows == 1)
  int32_t per;                 // units a workgroup takes of a row (rows == 1)
};

__device__ __forceinline__ float2 cos_sin(int32_t position, float freq) {
  const double t = (double)position * (double)freq;
  const double t_rest = __builtin_fma((double)position, (double)freq, -t);
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;   // 1 / (2 pi)
  const double hi = t * kHi;
  const double lo = __builtin_fma(t_rest, kHi, __builtin_fma(t, kLo, __builtin_fma(t, kHi, -hi)));
  const double quarter = __builtin_rint(4.0 * hi);
  const double rest = __builtin_fma(-0.25, quarter, hi) + lo;   // turns
  float s, c;
  sincospif((float)(2.0 * rest), &s, &c);
  const int k = (int)(quarter - 4.0 * __builtin_floor(0.25 * quarter));
  const float cc = (k & 1) ? s : c, ss = (k & 1) ? c : s;
  return {(k == 1 || k == 2) ? -cc : cc, (k & 2) ? -ss : ss};
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a, RopeTile t) {
  extern __shared__ float2 s_turn[];   // [rows][rotary / 2]
  const int half = a.rotary / 2;
  const int64_t row0 = t.rows == 1 ? blockIdx.x / t.parts : (int64_t)blockIdx.x * t.rows;
  const int part = t.rows == 1 ? (int)(blockIdx.x % t.parts) : 0;
  const int rows = (int)(a.rows - row0 < t.rows ? a.rows - row0 : t.rows);
  for (int i = threadIdx.x; i < rows * half; i += kRopeThreads) {
    const int r = i / half;
    const float2 cs = cos_sin(a.positions[row0 + r], a.inv_freq[i - r * half]);
    s_turn[i] = {cs.x * a.scale, cs.y * a.scale};
  }
  __syncthreads();
  const int first = part * t.per;
  const int end = t.rows == 1 ? min(t.units, first + t.per) : rows * t.units;
  for (int i = first + threadIdx.x; i < end; i += kRopeThreads) {
    const int r = i / t.units;
    int u = i - r * t.units;
    const bool is_k = u >= t.q_units;
    u -= is_k ? t.q_units : 0;
    const int head = u / t.head_units;
    u -= head * t.head_units;
    const int64_t row = row0 + r;
    const uint16_t* from = (is_k ? a.k + row * a.k_stride : a.q + row * a.q_stride) + head * a.dim;
    uint16_t* to = (is_k ? a.k_out + row * a.k_out_stride : a.q_out + row * a.q_out_stride) + head * a.dim;
    // two pieces of 8 dimensions: the pairs' halves, or (adjacent pairs, and dimensions that stay) 16 in a row
    const bool turn = u < t.turned;
    const int lo = !INTERLEAVED && turn ? 8 * u : 16 * u, hi = !INTERLEAVED && turn ? half + 8 * u : 16 * u + 8;
    u32x4 v = *reinterpret_cast<const u32x4*>(from + lo), w = *reinterpret_cast<const u32x4*>(from + hi);
    if (turn) {
      const float2* cs = s_turn + r * half + 8 * u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (INTERLEAVED) {
          const float2 c0 = cs[j], c1 = cs[4 + j];
          const float a0 = bf16_to_f32(v[j] & 0xFFFFu), b0 = __uint_as_float(v[j] & 0xFFFF0000u);
          const float a1 = bf16_to_f32(w[j] & 0xFFFFu), b1 = __uint_as_float(w[j] & 0xFFFF0000u);
          v[j] = bf16_rne(__builtin_fmaf(a0, c0.x, -(b0 * c0.y))) |
                 ((uint32_t)bf16_rne(__builtin_fmaf(b0, c0.x, a0 * c0.y)) << 16);
          w[j] = bf16_rne(__builtin_fmaf(a1, c1.x, -(b1 * c1.y))) |
                 ((uint32_t)bf16_rne(__builtin_fmaf(b1, c1.x, a1 * c1.y)) << 16);
        } else {
          const float2 c0 = cs[2 * j], c1 = cs[2 * j + 1];
          const float a0 = bf16_to_f32(v[j] & 0xFFFFu), a1 = __uint_as_float(v[j] & 0xFFFF0000u);
          const float b0 = bf16_to_f32(w[j] & 0xFFFFu), b1 = __uint_as_float(w[j] & 0xFFFF0000u);
          v[j] = bf16_rne(__builtin_fmaf(a0, c0.x, -(b0 * c0.y))) |
                 ((uint32_t)bf16_rne(__builtin_fmaf(a1, c1.x, -(b1 * c1.y))) << 16);
          w[j] = bf16_rne(__builtin_fmaf(b0, c0.x, a0 * c0.y)) |
                 ((uint32_t)bf16_rne(__builtin_fmaf(b1, c1.x, a1 * c1.y)) << 16);
        }
      }
    }
    *reinterpret_cast<u32x4*>(to + lo) = v;
    *reinterpret_cast<u32x4*>(to + hi) = w;
  }
}

}  // namespace

void launch_rope(const RopeArgs& a, bool interleaved, hipStream_t stream) {
  RopeTile t{};
  t.head_units = a.dim / 16;
  t.turned = a.rotary / 16;
  t.q_units = a.q_heads * t.head_units;
  t.units = t.q_units + a.k_heads * t.head_units;
  t.per = a.rows * t.units > kFewUnits ? 2 * kRopeThreads : kRopeThreads;
  t.rows = t.units >= t.per ? 1 : min(16, t.per / t.units);
  t.parts = t.rows == 1 ? (t.units + t.per - 1) / t.per : 1;
  const size_t lds = (size_t)t.rows * (a.rotary / 2) * sizeof(float2);
  // a launch holds fewer than 2^32 threads
  const int64_t slice = ((int64_t)1 << 23) / t.parts * t.rows;
  for (int64_t r0 = 0; r0 < a.rows; r0 += slice) {
    RopeArgs s = a;
    s.rows = a.rows - r0 < slice ? a.rows - r0 : slice;
    s.positions += r0;
    s.q += r0 * a.q_stride;
    s.q_out += r0 * a.q_out_stride;
    if (a.k) {
      s.k += r0 * a.k_stride;
      s.k_out += r0 * a.k_out_stride;
    }
    const unsigned grid = (unsigned)(t.rows == 1 ? s.rows * t.parts : (s.rows + t.rows - 1) / t.rows);
    if (interleaved) rope_kernel<true><<<grid, kRopeThreads, lds, stream>>>(s, t);
    else rope_kernel<false><<<grid, kRopeThreads, lds, stream>>>(s, t);
  }
}

}  // namespace w4
