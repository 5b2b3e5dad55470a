// Residual addition and RMS norm, with a bf16 or an E4M3 output.
//
//   r = bf16(x + residual)            (fp32 sum; r = x without a residual)
//   n = r * w',  w' = fl32(offset + weight)
//   y = n / sqrt(mean(r^2) + eps)
//   bf16 form: bf16(y).   E4M3 form: s = fl32(max|y| / 448) (1 where that is
//   0), code = E4M3(clamp(fl32(y / s), +-448)).
//
// A row's values are small multiples of one another, so many quotients by the
// row's scale fall on or next to the middle between two E4M3 values, and a
// statistic that is off in its 24th bit would decide those codes.  So the sum
// of squares is 64-bit, max|n| is taken of exact products, 1 / rms and s
// follow in 64 bits, and the per-element factor f (1 / rms, or 1 / (rms s))
// enters as two fp32 terms: r f = a + b with a = fl(r fh), b = fl(r fh - a +
// r fl), and y = fma(a, w', b w'), good to about 2^-46 before its rounding to
// fp32 (the bf16 form then rounds that to bf16).  That holds where neither r f
// nor its last bits leave fp32's range beside their w': rows whose statistics
// do, and chunks with a |w'| over 2^8 (or one that is not finite), take the same
// steps in 64 bits.
//
// Bound by memory for many rows (4096 x 2816 with residual, E4M3: 18.0 us, 4.5
// TB/s; 8191 x 4096 bf16: 23.4 us, 5.7 TB/s), by latency for few (one row 2.8
// us, 64 rows 4.2).  With the per-element arithmetic in 64 bits too they took
// 22.2, 29.1, 2.9 and 4.5 us.  A workgroup takes a row; a wave alone, holding
// 6 or 8 chunks a lane, was slower (22.4 us, and spilling).

#include "common.h"
#include "decode.h"
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
  double inv_d, eps;
  float offset;
  uint16_t* sum_out;          // nullable
  uint16_t* y;                // bf16 form
  uint8_t* q;                 // E4M3 form
  float* scale;
};

// One 16-byte chunk: r as bf16 pairs.
__device__ __forceinline__ u32x4 chunk_sum(u32x4 v, u32x4 e) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = bf16_to_f32(v[i] & 0xFFFFu) + bf16_to_f32(e[i] & 0xFFFFu);
    const float hi = __uint_as_float(v[i] & 0xFFFF0000u) + __uint_as_float(e[i] & 0xFFFF0000u);
    v[i] = (uint32_t)bf16_rne(lo) | ((uint32_t)bf16_rne(hi) << 16);
  }
  return v;
}

__device__ __forceinline__ float chunk_value(u32x4 v, int i) {
  return (i & 1) ? __uint_as_float(v[i >> 1] & 0xFFFF0000u) : bf16_to_f32(v[i >> 1] & 0xFFFFu);
}

__device__ __forceinline__ double scaled(u32x4 r, u32x4 w, int i, float offset) {
  return (double)chunk_value(r, i) * (double)(chunk_value(w, i) + offset);
}

template <int CTRL>
__device__ __forceinline__ double dpp_row_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double lane_f64(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Over the wave; every lane gets the result.
__device__ __forceinline__ double wave_sum_f64(double v) {
  v += dpp_row_f64<0xB1>(v);
  v += dpp_row_f64<0x4E>(v);
  v += dpp_row_f64<0x141>(v);
  v += dpp_row_f64<0x140>(v);
  return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}
// v >= 0, or a NaN as the largest bit pattern: compared as integers
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const uint64_t w = ((uint64_t)(uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), o, 64) << 32) |
                       (uint32_t)__shfl_xor((int)(uint32_t)v, o, 64);
    v = w > v ? w : v;
  }
  return v;
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max_u32<0x140>(dpp_max_u32<0x141>(dpp_max_u32<0x4E>(dpp_max_u32<0xB1>(v))));
  return max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
             max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

// Whether every |w'| of the chunk is at most 2^8: what r f loses below 2^-149 is
// then at most 2^-141 in y, less than fp32's rounding of a y from 2^-117 up, and
// 2^-8 of bf16's smallest step.
__device__ __forceinline__ bool weights_near_one(u32x4 w, float offset) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
  return bf16_to_f32(max(m[0], m[1])) + __builtin_fabsf(offset) <= 256.0f;   // not for a NaN
}

// The output factor of a row: f = fh + fl, or (wide) in 64 bits.
struct Factor {
  float fh, fl;
  double f;
  bool wide;      // the two fp32 terms may leave their range
  bool poison;    // E4M3: a NaN or an infinity in the row
};

template <bool QUANT>
__device__ __forceinline__ void store_chunk(const NormArgs& a, int64_t row, int ch, u32x4 r, u32x4 w, const Factor& k) {
  float y[8];
  if (!k.wide && weights_near_one(w, a.offset)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = chunk_value(r, i), t = chunk_value(w, i) + a.offset;
      const float p = v * k.fh;
      const float q = __builtin_fmaf(v, k.fl, __builtin_fmaf(v, k.fh, -p));
      y[i] = __builtin_fmaf(p, t, q * t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = k.poison ? 0.f : (float)(scaled(r, w, i, a.offset) * k.f);
  }
  if constexpr (QUANT) {
    u32x2 o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = fminf(fmaxf(y[4 * h + i], -448.0f), 448.0f);
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
      p = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], p, true);
      o[h] = (uint32_t)p;
    }
    reinterpret_cast<u32x2*>(a.q + row * a.d)[ch] = o;
  } else {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f32_to_bf16(y[2 * i]) | (f32_to_bf16(y[2 * i + 1]) << 16);
    reinterpret_cast<u32x4*>(a.y + row * a.d)[ch] = o;
  }
}

// TPR threads per row (64 or 256).  NCH > 0: at most NCH chunks per thread,
// kept in registers between the statistics and the output; NCH = 0: any d, r
// read again.  OFFSET: w' is not a bf16 value, so the products n need 64 bits.
template <int TPR, int NCH, bool QUANT, bool OFFSET>
__global__ void __launch_bounds__(kNormThreads) add_rmsnorm_kernel(NormArgs a) {
  constexpr int ROWS = kNormThreads / TPR;
  __shared__ double s_sum[4];
  __shared__ uint64_t s_max[4];
  const int tid = threadIdx.x % TPR, wv = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * ROWS + (TPR == 64 ? wv : 0);
  if (TPR == 64 && row >= a.rows) return;
  const int nch = a.d / 8;
  const u32x4* xs = reinterpret_cast<const u32x4*>(a.x + row * a.d);
  const u32x4* es = reinterpret_cast<const u32x4*>(a.residual ? a.residual + row * a.d : nullptr);
  const u32x4* ws = reinterpret_cast<const u32x4*>(a.weight);
  u32x4* sums = reinterpret_cast<u32x4*>(a.sum_out ? a.sum_out + row * a.d : nullptr);
  // r a second time: from sum_out where it was stored (x or the residual may
  // be the same memory), else from the inputs
  auto row_again = [&](int ch) { return sums ? sums[ch] : es ? chunk_sum(xs[ch], es[ch]) : xs[ch]; };
  double ss = 0.0;
  uint32_t top = 0;       // max |n| as bits: fp32 (exact unless OFFSET),
  uint64_t top64 = 0;     // or 64-bit
  auto stats = [&](u32x4 r, u32x4 w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = chunk_value(r, i);
      ss = __builtin_fma((double)v, (double)v, ss);
      if constexpr (QUANT && !OFFSET) top = max(top, __float_as_uint(v * chunk_value(w, i)) & 0x7FFFFFFFu);
      if constexpr (QUANT && OFFSET) {
        const uint64_t n = __builtin_bit_cast(uint64_t, __builtin_fabs(scaled(r, w, i, a.offset)));
        top64 = n > top64 ? n : top64;
      }
    }
  };
  u32x4 r[NCH > 0 ? NCH : 1], w[NCH > 0 ? NCH : 1];
  const u32x4 zero = {0u, 0u, 0u, 0u};
  if constexpr (NCH > 0) {
    u32x4 e[NCH];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int ch = tid + TPR * k;
      r[k] = e[k] = w[k] = zero;
      if (ch < nch) {
        r[k] = xs[ch];
        if (es) e[k] = es[ch];
        w[k] = ws[ch];
      }
    }
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int ch = tid + TPR * k;
      if (es) r[k] = chunk_sum(r[k], e[k]);
      if (sums && ch < nch) sums[ch] = r[k];
      if (ch < nch) stats(r[k], w[k]);
    }
  } else {
    for (int ch = tid; ch < nch; ch += TPR) {
      const u32x4 v = es ? chunk_sum(xs[ch], es[ch]) : xs[ch];
      if (sums) sums[ch] = v;
      stats(v, ws[ch]);
    }
  }
  ss = wave_sum_f64(ss);
  if constexpr (QUANT && !OFFSET) top = wave_max_u32(top);
  if constexpr (QUANT && OFFSET) top64 = wave_max_u64(top64);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) {
      s_sum[wv] = ss;
      s_max[wv] = OFFSET ? top64 : top;
    }
    __syncthreads();
    ss = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
    if constexpr (QUANT && !OFFSET)
      top = max(max((uint32_t)s_max[0], (uint32_t)s_max[1]), max((uint32_t)s_max[2], (uint32_t)s_max[3]));
    if constexpr (QUANT && OFFSET) {
#pragma unroll
      for (int i = 0; i < 4; ++i) top64 = s_max[i] > top64 ? s_max[i] : top64;
    }
  }

  Factor k{};
  const double ms = ss * a.inv_d + a.eps;
  // 1 / sqrt(ms): the hardware's estimate and two Newton steps, or the slow way
  // where an element's fp32 terms could leave the normal range
  k.wide = !(ms > 0x1p-80 && ms < 0x1p80);
  double rstd;
  if (!k.wide) {
    rstd = __builtin_amdgcn_rsq(ms);
    rstd = rstd * __builtin_fma(-0.5 * ms * rstd, rstd, 1.5);
    rstd = rstd * __builtin_fma(-0.5 * ms * rstd, rstd, 1.5);
  } else {
    rstd = 1.0 / __builtin_sqrt(ms);
  }
  k.f = rstd;
  if constexpr (QUANT) {
    double m;
    if constexpr (OFFSET) {
      m = __builtin_bit_cast(double, top64);
    } else {
      m = (double)__uint_as_float(top);
      if (!(m > 0x1p-80 && m < 0x1p120)) {
        // products below fp32's normal range or above it (or not finite): taken again in 64 bits
        top64 = 0;
        auto again = [&](u32x4 rv, u32x4 wvv) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint64_t n = __builtin_bit_cast(uint64_t, __builtin_fabs(scaled(rv, wvv, i, a.offset)));
            top64 = n > top64 ? n : top64;
          }
        };
        if constexpr (NCH > 0) {
#pragma unroll
          for (int i = 0; i < NCH; ++i) again(r[i], w[i]);
        } else {
          for (int ch = tid; ch < nch; ch += TPR) again(row_again(ch), ws[ch]);
        }
        top64 = wave_max_u64(top64);
        if constexpr (TPR > 64) {
          __syncthreads();   // s_max read above
          if ((threadIdx.x & 63) == 0) s_max[wv] = top64;
          __syncthreads();
#pragma unroll
          for (int i = 0; i < 4; ++i) top64 = s_max[i] > top64 ? s_max[i] : top64;
        }
        m = __builtin_bit_cast(double, top64);
        k.wide = true;
      }
    }
    m *= rstd;
    float s = (float)(m * (1.0 / 448.0));
    k.poison = !(m < __builtin_inf()) || !(s < INFINITY);
    if (s == 0.f) s = 1.0f;
    k.wide |= k.poison || !(s > 0x1p-80f && s < 0x1p80f);
    k.f = rstd / (double)s;
    if (tid == 0) a.scale[row] = k.poison ? __uint_as_float(0x7FC00000u) : s;
  }
  k.fh = (float)k.f;
  k.fl = (float)(k.f - (double)k.fh);
  if constexpr (NCH > 0) {
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (tid + TPR * i < nch) store_chunk<QUANT>(a, row, tid + TPR * i, r[i], w[i], k);
  } else {
    for (int ch = tid; ch < nch; ch += TPR)
      store_chunk<QUANT>(a, row, ch, row_again(ch), ws[ch], k);
  }
}

// Rows of up to 1024 values leave lanes of a workgroup idle: a wave takes one
// (32768 x 1024 bf16: 51.7 against 60.7 us, 65536 x 512 E4M3: 50.5 against
// 93.4).  The rule does not look at the number of rows; few of them would be
// faster by workgroups (8 rows of 1024: 3.0 against 3.6 us).
constexpr int kWaveChunks = 128;

template <bool QUANT, bool OFFSET>
void launch_norm(const NormArgs& a, hipStream_t stream) {
  const int nch = a.d / 8;
  if (nch <= kWaveChunks) {
    const dim3 grid((unsigned)((a.rows + 3) / 4));
    if (nch <= 64) add_rmsnorm_kernel<64, 1, QUANT, OFFSET><<<grid, kNormThreads, 0, stream>>>(a);
    else add_rmsnorm_kernel<64, 2, QUANT, OFFSET><<<grid, kNormThreads, 0, stream>>>(a);
    return;
  }
  const dim3 grid((unsigned)a.rows);
  const int per = (nch + kNormThreads - 1) / kNormThreads;
  if (per <= 1) add_rmsnorm_kernel<256, 1, QUANT, OFFSET><<<grid, kNormThreads, 0, stream>>>(a);
  else if (per <= 2) add_rmsnorm_kernel<256, 2, QUANT, OFFSET><<<grid, kNormThreads, 0, stream>>>(a);
  else if (per <= 4) add_rmsnorm_kernel<256, 4, QUANT, OFFSET><<<grid, kNormThreads, 0, stream>>>(a);
  else add_rmsnorm_kernel<256, 0, QUANT, OFFSET><<<grid, kNormThreads, 0, stream>>>(a);
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
               1.0 / (double)d, (double)eps, offset, sum_out ? sum_out + at : nullptr, y ? y + at : nullptr,
               q ? q + at : nullptr, scale ? scale + r0 : nullptr};
    const bool add = offset != 0.f;   // (a NaN offset too)
    if (!q) launch_norm<false, false>(a, stream);
    else if (add) launch_norm<true, true>(a, stream);
    else launch_norm<true, false>(a, stream);
  }
}

}  // namespace w4
