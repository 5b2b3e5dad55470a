// Residual addition and RMS norm, with a bf16 or an E4M3 output.
//
//   r = bf16(x + residual)            (fp32 sum; r = x without a residual)
//   n = r * w',  w' = fl32(offset + weight)
//   y = n / sqrt(mean(r^2) + eps)
//   bf16 form: bf16(y).   E4M3 form: s = fl32(max|y| / 448) (1 where that is
//   0), code = E4M3(clamp(fl32(y / s), +-448)).
//
// The sum of squares, n (an exact product: 8 by 24 bits), y and y / s are
// 64-bit.  A row's values are small multiples of one another, so many
// quotients by the row's scale fall on or next to the middle between two E4M3
// values: with 32-bit intermediates the order of the additions would decide
// those codes.  The 64-bit operations run at the fp32 rate here and the kernel
// waits for memory either way.

#include "common.h"
#include "internal.h"
#include "w4a16.h"

namespace w4 {

namespace {

constexpr int kNormThreads = 256;

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;   // nullable
  const uint16_t* weight;
  int64_t rows;
  int d;
  double eps;
  float offset;
  uint16_t* sum_out;          // nullable
  uint16_t* y;                // bf16 form
  uint8_t* q;                 // E4M3 form
  float* scale;
};

// One 16-byte chunk: r as bf16 pairs (stored to sum_out if wanted).
__device__ __forceinline__ u32x4 norm_chunk_sum(const NormArgs& a, int64_t row, int ch) {
  u32x4 v = reinterpret_cast<const u32x4*>(a.x + row * a.d)[ch];
  if (a.residual) {
    const u32x4 e = reinterpret_cast<const u32x4*>(a.residual + row * a.d)[ch];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = f32_to_bf16(bf16_to_f32(v[i] & 0xFFFFu) + bf16_to_f32(e[i] & 0xFFFFu));
      const uint32_t hi = f32_to_bf16(bf16_to_f32(v[i] >> 16) + bf16_to_f32(e[i] >> 16));
      v[i] = lo | (hi << 16);
    }
  }
  return v;
}

__device__ __forceinline__ float chunk_value(u32x4 v, int i) {
  return (i & 1) ? __uint_as_float(v[i >> 1] & 0xFFFF0000u) : bf16_to_f32(v[i >> 1] & 0xFFFFu);
}

// n of element i of a chunk
__device__ __forceinline__ double scaled(u32x4 r, u32x4 w, int i, float offset) {
  return (double)chunk_value(r, i) * (double)(chunk_value(w, i) + offset);
}

template <bool QUANT>
__device__ __forceinline__ void store_chunk(const NormArgs& a, int64_t row, int ch, u32x4 r, u32x4 w, double f) {
  if constexpr (QUANT) {
    u32x2 o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        t[i] = fminf(fmaxf((float)(scaled(r, w, 4 * h + i, a.offset) * f), -448.0f), 448.0f);
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
      p = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], p, true);
      o[h] = (uint32_t)p;
    }
    reinterpret_cast<u32x2*>(a.q + row * a.d)[ch] = o;
  } else {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = f32_to_bf16((float)(scaled(r, w, 2 * i, a.offset) * f));
      const uint32_t hi = f32_to_bf16((float)(scaled(r, w, 2 * i + 1, a.offset) * f));
      o[i] = lo | (hi << 16);
    }
    reinterpret_cast<u32x4*>(a.y + row * a.d)[ch] = o;
  }
}

__device__ __forceinline__ double shfl_xor_f64(double v, int o) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)b, o, 64);
  const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(b >> 32), o, 64);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// One workgroup per row.  NCH > 0: at most NCH chunks per thread, kept in
// registers between the statistics and the output; NCH = 0: any d, r re-read.
template <int NCH, bool QUANT>
__global__ void __launch_bounds__(kNormThreads) add_rmsnorm_kernel(NormArgs a) {
  __shared__ double s_sum[4], s_max[4];
  __shared__ int s_bad[4];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t row = blockIdx.x;
  const int nch = a.d / 8;
  const u32x4* wsrc = reinterpret_cast<const u32x4*>(a.weight);
  u32x4 r[NCH > 0 ? NCH : 1], w[NCH > 0 ? NCH : 1];
  double ss = 0.0, top = 0.0;
  bool bad = false;
  auto take = [&](u32x4 rv, u32x4 wvv, int ch) {
    if (a.sum_out) reinterpret_cast<u32x4*>(a.sum_out + row * a.d)[ch] = rv;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double f = (double)chunk_value(rv, i);
      ss = __builtin_fma(f, f, ss);
      if constexpr (QUANT) {
        const double n = __builtin_fabs(scaled(rv, wvv, i, a.offset));
        bad |= !(n < __builtin_inf());
        top = __builtin_fmax(top, n);
      }
    }
  };
  if constexpr (NCH > 0) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int ch = threadIdx.x + kNormThreads * k;
      r[k] = u32x4{0u, 0u, 0u, 0u};
      w[k] = r[k];
      if (ch < nch) {
        r[k] = norm_chunk_sum(a, row, ch);
        w[k] = wsrc[ch];
      }
    }
#pragma unroll
    for (int k = 0; k < NCH; ++k)
      if (threadIdx.x + kNormThreads * k < nch) take(r[k], w[k], threadIdx.x + kNormThreads * k);
  } else {
    for (int ch = threadIdx.x; ch < nch; ch += kNormThreads) take(norm_chunk_sum(a, row, ch), wsrc[ch], ch);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    ss += shfl_xor_f64(ss, o);
    if constexpr (QUANT) top = __builtin_fmax(top, shfl_xor_f64(top, o));
  }
  const int any_bad = QUANT ? (__ballot(bad) != 0) : 0;
  if (lane == 0) {
    s_sum[wv] = ss;
    s_max[wv] = top;
    s_bad[wv] = any_bad;
  }
  __syncthreads();
  ss = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
  const double rstd = 1.0 / __builtin_sqrt(ss / (double)a.d + a.eps);
  double f = rstd;
  bool poison = false;
  if constexpr (QUANT) {
    top = __builtin_fmax(__builtin_fmax(s_max[0], s_max[1]), __builtin_fmax(s_max[2], s_max[3])) * rstd;
    poison = (s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3]) || !(top < __builtin_inf());
    float s = (float)(top / 448.0);
    if (s == 0.f) s = 1.0f;
    if (!(s < INFINITY)) poison = true;
    f = rstd / (double)s;
    if (threadIdx.x == 0) a.scale[row] = poison ? __uint_as_float(0x7FC00000u) : s;
  }
  // a row that holds a NaN or an infinity: codes 0 under a NaN scale
  const u32x4 zero = {0u, 0u, 0u, 0u};
  if constexpr (NCH > 0) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int ch = threadIdx.x + kNormThreads * k;
      if (ch < nch) store_chunk<QUANT>(a, row, ch, poison ? zero : r[k], poison ? zero : w[k], poison ? 0.0 : f);
    }
  } else {
    for (int ch = threadIdx.x; ch < nch; ch += kNormThreads) {
      // r again: from sum_out where it was stored (x or the residual may be
      // the same memory), else from the inputs
      const u32x4 rv = a.sum_out ? reinterpret_cast<const u32x4*>(a.sum_out + row * a.d)[ch] : norm_chunk_sum(a, row, ch);
      store_chunk<QUANT>(a, row, ch, poison ? zero : rv, poison ? zero : wsrc[ch], poison ? 0.0 : f);
    }
  }
}

template <bool QUANT>
void launch_norm_t(const NormArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.rows), block(kNormThreads);
  const int per = (a.d / 8 + kNormThreads - 1) / kNormThreads;
  if (per <= 1) add_rmsnorm_kernel<1, QUANT><<<grid, block, 0, stream>>>(a);
  else if (per <= 2) add_rmsnorm_kernel<2, QUANT><<<grid, block, 0, stream>>>(a);
  else if (per <= 4) add_rmsnorm_kernel<4, QUANT><<<grid, block, 0, stream>>>(a);
  else add_rmsnorm_kernel<0, QUANT><<<grid, block, 0, stream>>>(a);
}

}  // namespace

void launch_add_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t rows, int64_t d,
                        float eps, float offset, uint16_t* sum_out, uint16_t* y, uint8_t* q, float* scale,
                        hipStream_t stream) {
  // a launch holds fewer than 2^32 threads
  constexpr int64_t kSlice = (int64_t)1 << 22;
  for (int64_t r0 = 0; r0 < rows; r0 += kSlice) {
    const int64_t at = r0 * d;
    NormArgs a{x + at, residual ? residual + at : nullptr, weight, rows - r0 < kSlice ? rows - r0 : kSlice, (int)d,
               (double)eps, offset, sum_out ? sum_out + at : nullptr, y ? y + at : nullptr, q ? q + at : nullptr,
               scale ? scale + r0 : nullptr};
    if (q) launch_norm_t<true>(a, stream);
    else launch_norm_t<false>(a, stream);
  }
}

}  // namespace w4
