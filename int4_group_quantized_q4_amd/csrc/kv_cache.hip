// Writing new tokens' keys and values into the paged cache, quantized on the
// way, and reading rows back.
//
// Bound by the bytes of the rows on one side and of the cache on the other:
// every row is read once and written once.  A group of TP lanes takes one
// (token, head) row, 8 dimensions a lane, so that a row is one contiguous
// load, its scale a few cross-lane maxima, and its codes stay in registers.

#include "common.h"
#include "internal.h"
#include "kv_layout.h"
#include "w4a16.h"

namespace w4 {

namespace {

constexpr int kThreads = 256;

template <int NG>
struct RowSplit {
  static constexpr int CH = 4 * NG;                    // 8-dimension chunks of a row
  static constexpr int TP = CH < 16 ? CH : 16;         // lanes per row
  static constexpr int CPT = CH / TP;                  // chunks per lane
  static constexpr int ROWS = kThreads / TP;           // rows per workgroup
};

// maximum over aligned groups of N lanes (N = 4, 8 or 16)
template <int N>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

__device__ __forceinline__ uint32_t max_magnitude(u32x4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = max(m, v[i] & 0x7FFFu);
    m = max(m, (v[i] >> 16) & 0x7FFFu);
  }
  return m;
}

__device__ __forceinline__ float value_of(u32x4 v, int i) {
  return (i & 1) ? __uint_as_float(v[i >> 1] & 0xFFFF0000u) : bf16_to_f32(v[i >> 1] & 0xFFFFu);
}

constexpr uint32_t kInfBits = 0x7F80u;   // bf16 magnitudes from here up: infinity, NaN

struct Row {
  int64_t page;
  int tile, r;   // tile in the page, token in the tile
};

// The row of a slot; false for padding and for slots outside the cache.
__device__ __forceinline__ bool find_row(int64_t slot, const KvArgs& a, Row& o) {
  if (slot < 0 || slot >= a.n_pages << a.page_shift) return false;
  const int in_page = (int)(slot & ((1 << a.page_shift) - 1));
  o.page = slot >> a.page_shift;
  o.tile = in_page / kKvTile;
  o.r = in_page % kKvTile;
  return true;
}

template <int FMT, int NG, bool V>
__device__ void write_rows(const KvArgs& a) {
  typedef KvLayout<FMT, NG> L;
  typedef RowSplit<NG> S;
  const int64_t tok = (int64_t)blockIdx.x * S::ROWS + threadIdx.x / S::TP;
  const int m = threadIdx.x % S::TP;
  const int head = blockIdx.y;
  Row row{};
  bool live = false;
  if (tok < a.tokens) {
    const int64_t slot = a.slots[tok];
    live = find_row(slot, a, row);
    if (!V && !live && slot >= 0 && head == 0 && m == 0 && a.counters) atomicAdd(a.counters, 1ull);
  }
  const uint16_t* src = V ? a.v + tok * a.v_stride : a.k + tok * a.k_stride;
  u32x4 x[S::CPT];
#pragma unroll
  for (int i = 0; i < S::CPT; ++i) {
    x[i] = u32x4{0u, 0u, 0u, 0u};
    if (live) x[i] = *reinterpret_cast<const u32x4*>(src + (int64_t)head * L::D + 8 * (m + S::TP * i));
  }
  uint8_t* block = a.cache + row.page * a.page_bytes + (int64_t)head * 2 * a.block_bytes + (V ? a.block_bytes : 0);
  uint8_t* codes = block + (int64_t)row.tile * L::kTileBytes;
  uint8_t* scales = block + ((int64_t)L::kTileBytes << a.page_shift) / kKvTile + row.tile * L::kScaleTileBytes;
  uint32_t row_max = 0;
  if constexpr (FMT == W4_KV_E4M3) {
#pragma unroll
    for (int i = 0; i < S::CPT; ++i) row_max = max(row_max, max_magnitude(x[i]));
    row_max = group_max<S::TP>(row_max);
  }
#pragma unroll
  for (int i = 0; i < S::CPT; ++i) {
    const int ch = m + S::TP * i, g = ch >> 2, c = ch & 3;   // dimensions 32g + 8c ..
    const int unit = g / L::U, part = g % L::U;
    // where a K row keeps these 8 dimensions: lane 16c + r of the unit
    uint8_t* kdst = codes + (unit * 64 + 16 * c + row.r) * L::kUnitBytes + part * L::kGroupBytes;
    // V: dimension 32g + 8c + 2t + b sits in lane 16*(r/4) + 4c + t, at [b][r%4]
    uint8_t* vdst = codes + (unit * 64 + 16 * (row.r >> 2) + 4 * c) * L::kUnitBytes + part * L::kGroupBytes;
    const int j = row.r & 3;
    if constexpr (FMT == W4_KV_BF16) {
      if (!live) continue;
      if constexpr (!V) {
        *reinterpret_cast<u32x4*>(kdst) = x[i];
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint16_t* p = reinterpret_cast<uint16_t*>(vdst + t * L::kUnitBytes) + j;
          p[0] = (uint16_t)(x[i][t] & 0xFFFFu);
          p[4] = (uint16_t)(x[i][t] >> 16);
        }
      }
    } else if constexpr (FMT == W4_KV_E4M3) {
      const bool poison = row_max >= kInfBits;
      float s = bf16_to_f32(row_max) / 448.0f;
      if (s == 0.f) s = 1.0f;
      uint32_t w[2] = {0u, 0u};
      if (!poison) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float f[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) f[t] = fminf(fmaxf(value_of(x[i], 4 * h + t) / s, -448.0f), 448.0f);
          int p = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
          p = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], p, true);
          w[h] = (uint32_t)p;
        }
      }
      if (!live) continue;
      if (ch == 0) {
        reinterpret_cast<float*>(scales)[row.r] = poison ? __uint_as_float(0x7FC00000u) : s;
        if (poison && a.counters) atomicAdd(a.counters + 1, 1ull);
      }
      if constexpr (!V) {
        *reinterpret_cast<u32x2*>(kdst) = u32x2{w[0], w[1]};
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) vdst[(t >> 1) * L::kUnitBytes + 4 * (t & 1) + j] = (uint8_t)(w[t >> 2] >> (8 * (t & 3)));
      }
    } else {
      const uint32_t gm = group_max<4>(max_magnitude(x[i]));   // the 4 lanes of a group are adjacent
      const bool poison = gm >= kInfBits;
      const uint32_t sb = poison ? 0x7FC0u : f32_to_bf16(bf16_to_f32(gm) / 7.0f);
      const float s = bf16_to_f32(sb);
      uint32_t u[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        float q = 0.f;
        if (!poison && s > 0.f) q = fminf(fmaxf(rintf(value_of(x[i], t) / s), -8.0f), 7.0f);
        u[t] = (uint32_t)((int)q + 8);
      }
      if (!live) continue;
      if (c == 0) {
        reinterpret_cast<uint16_t*>(scales)[((row.r >> 2) * NG + g) * 4 + j] = (uint16_t)sb;
        if (poison && a.counters) atomicAdd(a.counters + 1, 1ull);
      }
      if constexpr (!V) {
        uint32_t w = 0;
#pragma unroll
        for (int t = 0; t < 8; ++t) w |= u[t] << tile16_bit(t);
        *reinterpret_cast<uint32_t*>(kdst) = w;
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) vdst[t * L::kUnitBytes + j] = (uint8_t)(u[2 * t] | (u[2 * t + 1] << 4));
      }
    }
  }
}

template <int FMT, int NG>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(KvArgs a) {
  if (blockIdx.z == 0) write_rows<FMT, NG, false>(a);
  else write_rows<FMT, NG, true>(a);
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0); }

template <int FMT, int NG, bool V, typename OUT>
__device__ void read_rows(const KvArgs& a) {
  typedef KvLayout<FMT, NG> L;
  typedef RowSplit<NG> S;
  const int64_t tok = (int64_t)blockIdx.x * S::ROWS + threadIdx.x / S::TP;
  if (tok >= a.tokens) return;
  const int m = threadIdx.x % S::TP;
  const int head = blockIdx.y;
  Row row{};
  const int64_t slot = a.slots[tok];
  if (!find_row(slot, a, row)) {
    if (!V && slot >= 0 && head == 0 && m == 0 && a.counters) atomicAdd(a.counters, 1ull);
    return;
  }
  const uint8_t* block = a.cache + row.page * a.page_bytes + (int64_t)head * 2 * a.block_bytes + (V ? a.block_bytes : 0);
  const uint8_t* codes = block + (int64_t)row.tile * L::kTileBytes;
  const uint8_t* scales = block + ((int64_t)L::kTileBytes << a.page_shift) / kKvTile + row.tile * L::kScaleTileBytes;
  OUT* dst = reinterpret_cast<OUT*>(V ? a.v_out : a.k_out) + tok * (V ? a.v_stride : a.k_stride) + (int64_t)head * L::D;
#pragma unroll
  for (int i = 0; i < S::CPT; ++i) {
    const int ch = m + S::TP * i, g = ch >> 2, c = ch & 3;
    const int unit = g / L::U, part = g % L::U;
    const uint8_t* ksrc = codes + (unit * 64 + 16 * c + row.r) * L::kUnitBytes + part * L::kGroupBytes;
    const uint8_t* vsrc = codes + (unit * 64 + 16 * (row.r >> 2) + 4 * c) * L::kUnitBytes + part * L::kGroupBytes;
    const int j = row.r & 3;
    float f[8];
    if constexpr (FMT == W4_KV_BF16) {
      if constexpr (!V) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(ksrc);
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] = value_of(w, t);
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
          f[t] = bf16_to_f32(reinterpret_cast<const uint16_t*>(vsrc + (t >> 1) * L::kUnitBytes)[4 * (t & 1) + j]);
      }
    } else if constexpr (FMT == W4_KV_E4M3) {
      const float s = reinterpret_cast<const float*>(scales)[row.r];
      if constexpr (!V) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(ksrc);
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] = s * e4m3_to_f32((w[t >> 2] >> (8 * (t & 3))) & 0xFFu);
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] = s * e4m3_to_f32(vsrc[(t >> 1) * L::kUnitBytes + 4 * (t & 1) + j]);
      }
    } else {
      const float s = bf16_to_f32(reinterpret_cast<const uint16_t*>(scales)[((row.r >> 2) * NG + g) * 4 + j]);
      if constexpr (!V) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(ksrc);
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] = s * (float)((int)((w >> tile16_bit(t)) & 0xFu) - 8);
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t b = vsrc[t * L::kUnitBytes + j];
          f[2 * t] = s * (float)((int)(b & 0xFu) - 8);
          f[2 * t + 1] = s * (float)((int)(b >> 4) - 8);
        }
      }
    }
    OUT* o = dst + 8 * ch;
    if constexpr (sizeof(OUT) == 4) {
      *reinterpret_cast<f32x4*>(o) = f32x4{f[0], f[1], f[2], f[3]};
      *reinterpret_cast<f32x4*>(o + 4) = f32x4{f[4], f[5], f[6], f[7]};
    } else {
      u32x4 w;
#pragma unroll
      for (int t = 0; t < 4; ++t) w[t] = f32_to_bf16(f[2 * t]) | (f32_to_bf16(f[2 * t + 1]) << 16);
      *reinterpret_cast<u32x4*>(o) = w;
    }
  }
}

template <int FMT, int NG, typename OUT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(KvArgs a) {
  if (blockIdx.z == 0) read_rows<FMT, NG, false, OUT>(a);
  else read_rows<FMT, NG, true, OUT>(a);
}

template <int FMT, int NG>
void launch_fmt(const KvArgs& a, bool write, int out_dtype, hipStream_t stream) {
  const dim3 grid((unsigned)((a.tokens + RowSplit<NG>::ROWS - 1) / RowSplit<NG>::ROWS), a.kv_heads, 2);
  if (write) kv_write_kernel<FMT, NG><<<grid, kThreads, 0, stream>>>(a);
  else if (out_dtype == W4_OUT_F32) kv_read_kernel<FMT, NG, float><<<grid, kThreads, 0, stream>>>(a);
  else kv_read_kernel<FMT, NG, uint16_t><<<grid, kThreads, 0, stream>>>(a);
}

template <int FMT>
void launch_dim(const KvArgs& a, bool write, int out_dtype, hipStream_t stream) {
  if (a.head_dim == 64) launch_fmt<FMT, 2>(a, write, out_dtype, stream);
  else if (a.head_dim == 128) launch_fmt<FMT, 4>(a, write, out_dtype, stream);
  else launch_fmt<FMT, 8>(a, write, out_dtype, stream);
}

void launch(const KvArgs& a, bool write, int out_dtype, hipStream_t stream) {
  if (a.format == W4_KV_BF16) launch_dim<W4_KV_BF16>(a, write, out_dtype, stream);
  else if (a.format == W4_KV_E4M3) launch_dim<W4_KV_E4M3>(a, write, out_dtype, stream);
  else launch_dim<W4_KV_Q4>(a, write, out_dtype, stream);
}

}  // namespace

void launch_kv_write(const KvArgs& a, hipStream_t stream) { launch(a, true, 0, stream); }
void launch_kv_read(const KvArgs& a, int out_dtype, hipStream_t stream) { launch(a, false, out_dtype, stream); }

}  // namespace w4
