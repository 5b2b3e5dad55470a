// Writing new tokens' keys and values into the paged cache, quantized on the
// way, and reading rows back.
//
// Bound by the bytes of the rows on one side and of the cache on the other:
// every row is read once and written once.  Four neighbouring lanes (a quad)
// take the same 8 dimensions of four consecutive tokens of the list, HB heads
// of K and of V each, all loads in flight together; so a wave reads whole
// rows, a row's scale is a few cross-lane maxima and its codes stay in
// registers.
//
// V lies in the cache as 4 tokens of one dimension side by side.  Where a
// quad's tokens are such a group (consecutive slots from a multiple of 4, as in
// a prompt), the quad exchanges its values (a 4 x 4 transpose, lane moves
// only) and each lane moves one wide piece; else each lane moves its token's
// single elements.  Reading 8192 consecutive E4M3 tokens of 8 x 128: 11.4 us
// exchanged, 17.2 us element by element; 30715 Q4 tokens of 4 x 256: 40 and 47
// us.  The rows read back leave by non-temporal stores, past the L2: 40 -> 29
// us (5.5 TB/s), 11.2 -> 9.8 us for the two.

#include "common.h"
#include "decode.h"
#include "kv_layout.h"
#include "w4a16.h"

namespace w4 {

namespace {

constexpr int kThreads = 256;

template <int NG>
struct RowSplit {
  static constexpr int CH = 4 * NG;                    // 8-dimension chunks of a row
  static constexpr int LP = CH < 16 ? CH : 16;         // lanes per row
  static constexpr int CPT = CH / LP;                  // chunks per lane
  static constexpr int ROWS = kThreads / LP;           // rows per workgroup
};

// maximum over the N lanes whose numbers differ in the bits from 4 up (a row's
// lanes are 4 apart)
template <int N>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
  for (int o = 4; o < 4 * N; o *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

// lane J of the quad's value
template <int J>
__device__ __forceinline__ uint32_t quad_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, J * 0x55, 0xF, 0xF, false);
}

// 4 x 4 transposes over a quad.  Dwords: lane q's x[i] <-> lane i's x[q].
__device__ __forceinline__ u32x4 quad_transpose(u32x4 x, int q) {
  const bool odd = q & 1, high = q & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {   // with the neighbour
    const uint32_t r = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(odd ? x[i] : x[i + 1]), 0xB1, 0xF, 0xF, false);
    x[i] = odd ? r : x[i];
    x[i + 1] = odd ? x[i + 1] : r;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {      // with the lane two on
    const uint32_t r = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(high ? x[i] : x[i + 2]), 0x4E, 0xF, 0xF, false);
    x[i] = high ? r : x[i];
    x[i + 2] = high ? x[i + 2] : r;
  }
  return x;
}
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
// Bytes: lane q's byte i <-> lane i's byte q.
__device__ __forceinline__ uint32_t quad_transpose_bytes(uint32_t x, int q) {
  const uint32_t sel = (uint32_t)q | ((uint32_t)(q + 4) << 8);
  const uint32_t p01 = __builtin_amdgcn_perm(quad_lane<1>(x), quad_lane<0>(x), sel);
  const uint32_t p23 = __builtin_amdgcn_perm(quad_lane<3>(x), quad_lane<2>(x), sel);
  return low_halves(p01, p23);
}
// Byte pairs: lane q's 8 bytes are pairs i (bytes 2i, 2i + 1); afterwards lane
// q holds pair q of lanes 0..3, first bytes in word 0, second in word 1.
__device__ __forceinline__ u32x2 quad_pairs_to_planes(u32x2 x, int q) {
  // every lane moves both words, then takes one (a lane move must not sit in a branch)
  const uint32_t a0 = quad_lane<0>(x[0]), a1 = quad_lane<1>(x[0]), a2 = quad_lane<2>(x[0]), a3 = quad_lane<3>(x[0]);
  const uint32_t b0 = quad_lane<0>(x[1]), b1 = quad_lane<1>(x[1]), b2 = quad_lane<2>(x[1]), b3 = quad_lane<3>(x[1]);
  const bool high = q & 2;
  const uint32_t w0 = high ? b0 : a0, w1 = high ? b1 : a1, w2 = high ? b2 : a2, w3 = high ? b3 : a3;
  const uint32_t b = 2u * (q & 1);   // [w0.b, w1.b, w0.b+1, w1.b+1]
  const uint32_t sel = b | ((b + 4) << 8) | ((b + 1) << 16) | ((b + 5) << 24);
  const uint32_t p01 = __builtin_amdgcn_perm(w1, w0, sel), p23 = __builtin_amdgcn_perm(w3, w2, sel);
  return u32x2{low_halves(p01, p23), high_halves(p01, p23)};
}
// The reverse.
__device__ __forceinline__ u32x2 quad_planes_to_pairs(u32x2 x, int q) {
  const uint32_t sel = (uint32_t)q | ((uint32_t)(q + 4) << 8);
  const uint32_t p0 = __builtin_amdgcn_perm(quad_lane<0>(x[1]), quad_lane<0>(x[0]), sel);
  const uint32_t p1 = __builtin_amdgcn_perm(quad_lane<1>(x[1]), quad_lane<1>(x[0]), sel);
  const uint32_t p2 = __builtin_amdgcn_perm(quad_lane<2>(x[1]), quad_lane<2>(x[0]), sel);
  const uint32_t p3 = __builtin_amdgcn_perm(quad_lane<3>(x[1]), quad_lane<3>(x[0]), sel);
  return u32x2{low_halves(p0, p1), low_halves(p2, p3)};
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

// x / s correctly rounded, as one IEEE division gives it, with r = fl32(1 / s)
// shared by a row or group: the product x r is within 2 steps of the quotient,
// one correction brings it within one, and a second one, from the then exact
// remainder, rounds it correctly (Markstein 1990).  Outside the range where no
// remainder is subnormal the division itself runs.
struct Divisor {
  float s, r;
  bool plain;
  __device__ __forceinline__ explicit Divisor(float d) : s(d), r(1.0f / d), plain(!(d > 0x1p-60f && d < 0x1p60f)) {}
  // the 8 values of a chunk, with one branch for all (one each: 9.1 against
  // 8.9 us for 4096 E4M3 tokens of 8 x 128, 6.2 against 5.9 for 2045 Q4 of 4 x 256)
  __device__ __forceinline__ void operator()(u32x4 x, float (&f)[8]) const {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float v = value_of(x, t);
      float q = v * r;
      q = __builtin_fmaf(__builtin_fmaf(-q, s, v), r, q);
      q = __builtin_fmaf(__builtin_fmaf(-q, s, v), r, q);
      f[t] = __builtin_copysignf(q, v);   // s > 0; the corrections would turn -0 into +0
    }
    if (plain) {
#pragma unroll
      for (int t = 0; t < 8; ++t) f[t] = value_of(x, t) / s;
    }
  }
};

constexpr uint32_t kInfBits = 0x7F80u;   // bf16 magnitudes from here up: infinity, NaN

// This lane's place in the list and the cache.
struct Place {
  int64_t tok;        // row of the list
  int64_t slot;
  int q, ch;          // lane of the quad, first chunk
  int tile, r;        // tile in the page, token in the tile
  const uint8_t* page;
  bool live;          // the slot lies in the cache
  bool quads;         // every quad of the wave holds 4 tokens side by side in the cache
};

template <int NG>
__device__ __forceinline__ Place find_place(const KvArgs& a) {
  typedef RowSplit<NG> S;
  Place p;
  const int lane = threadIdx.x & 63;
  p.q = lane & 3;
  p.ch = (lane >> 2) % S::LP;
  p.tok = (int64_t)blockIdx.x * S::ROWS + (threadIdx.x >> 6) * (64 / S::LP) + lane / (4 * S::LP) * 4 + p.q;
  p.slot = p.tok < a.tokens ? a.slots[p.tok] : -1;
  p.live = p.slot >= 0 && p.slot < a.n_pages << a.page_shift;
  const int64_t base = p.slot - p.q;
  const uint32_t lo = quad_lane<0>((uint32_t)base), hi = quad_lane<0>((uint32_t)(base >> 32));
  p.quads = __all(p.live && (p.slot & 3) == p.q && (uint32_t)base == lo && (uint32_t)(base >> 32) == hi);
  const int64_t slot = p.live ? p.slot : 0;
  const int in_page = (int)(slot & ((1 << a.page_shift) - 1));
  p.page = a.cache + (slot >> a.page_shift) * a.page_bytes;
  p.tile = in_page / kKvTile;
  p.r = in_page % kKvTile;
  return p;
}

// Where chunk ch (dimensions 32g + 8c ..) of a row keeps its codes in the
// tile: K: lane 16c + r of the group's unit.  V: dimension 32g + 8c + 2t + b in
// lane 16 (r/4) + 4c + t, element [b][r%4].
template <int FMT, int NG>
__device__ __forceinline__ uint32_t k_offset(int ch, int r) {
  typedef KvLayout<FMT, NG> L;
  const int g = ch >> 2, c = ch & 3;
  return (uint32_t)((g / L::U * 64 + 16 * c + r) * L::kUnitBytes + g % L::U * L::kGroupBytes);
}
template <int FMT, int NG>
__device__ __forceinline__ uint32_t v_offset(int ch, int r, int t) {
  typedef KvLayout<FMT, NG> L;
  const int g = ch >> 2, c = ch & 3;
  return (uint32_t)((g / L::U * 64 + 16 * (r >> 2) + 4 * c + t) * L::kUnitBytes + g % L::U * L::kGroupBytes);
}

// One head's K or V row piece(s) of this lane into the cache.
template <int FMT, int NG, bool V>
__device__ __forceinline__ void write_row(const KvArgs& a, const Place& pl, const u32x4 (&x)[RowSplit<NG>::CPT],
                                          int head) {
  typedef KvLayout<FMT, NG> L;
  typedef RowSplit<NG> S;
  uint8_t* block = const_cast<uint8_t*>(pl.page) + (int64_t)head * 2 * a.block_bytes + (V ? a.block_bytes : 0);
  uint8_t* codes = block + (uint32_t)pl.tile * (uint32_t)L::kTileBytes;
  uint8_t* scales = block + ((uint32_t)L::kTileBytes << a.page_shift) / kKvTile + pl.tile * L::kScaleTileBytes;
  const int j = pl.r & 3;
  uint32_t amax = 0;
  if constexpr (FMT == W4_KV_E4M3) {
#pragma unroll
    for (int i = 0; i < S::CPT; ++i) amax = max(amax, max_magnitude(x[i]));
    amax = row_max<S::LP>(amax);
  }
#pragma unroll
  for (int i = 0; i < S::CPT; ++i) {
    const int ch = pl.ch + S::LP * i, g = ch >> 2, c = ch & 3;
    if constexpr (FMT == W4_KV_BF16) {
      if constexpr (!V) {
        if (pl.live) *reinterpret_cast<u32x4*>(codes + k_offset<FMT, NG>(ch, pl.r)) = x[i];
      } else if (pl.quads) {
        // lane q: pairs q of the 4 tokens, as [b][j]
        const u32x4 y = quad_transpose(x[i], pl.q);
        const u32x4 w = {low_halves(y[0], y[1]), low_halves(y[2], y[3]), high_halves(y[0], y[1]),
                         high_halves(y[2], y[3])};
        *reinterpret_cast<u32x4*>(codes + v_offset<FMT, NG>(ch, pl.r, pl.q)) = w;
      } else if (pl.live) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint16_t* p = reinterpret_cast<uint16_t*>(codes + v_offset<FMT, NG>(ch, pl.r, t)) + j;
          p[0] = (uint16_t)(x[i][t] & 0xFFFFu);
          p[4] = (uint16_t)(x[i][t] >> 16);
        }
      }
    } else if constexpr (FMT == W4_KV_E4M3) {
      const bool poison = amax >= kInfBits;
      float s = bf16_to_f32(amax) / 448.0f;
      if (s == 0.f) s = 1.0f;
      const Divisor by(s);
      u32x2 w = {0u, 0u};
      float f[8];
      by(x[i], f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int t = 0; t < 4; ++t) f[4 * h + t] = __builtin_amdgcn_fmed3f(f[4 * h + t], -448.0f, 448.0f);
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h], f[4 * h + 1], 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2], f[4 * h + 3], p, true);
        w[h] = poison ? 0u : (uint32_t)p;
      }
      if (pl.live && ch == 0) {
        reinterpret_cast<float*>(scales)[pl.r] = poison ? __uint_as_float(0x7FC00000u) : s;
        if (poison && a.counters) atomicAdd(a.counters + 1, 1ull);
      }
      if constexpr (!V) {
        if (pl.live) *reinterpret_cast<u32x2*>(codes + k_offset<FMT, NG>(ch, pl.r)) = w;
      } else if (pl.quads) {
        *reinterpret_cast<u32x2*>(codes + v_offset<FMT, NG>(ch, pl.r, pl.q)) = quad_pairs_to_planes(w, pl.q);
      } else if (pl.live) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
          codes[v_offset<FMT, NG>(ch, pl.r, t >> 1) + 4 * (t & 1) + j] = (uint8_t)(w[t >> 2] >> (8 * (t & 3)));
      }
    } else {
      const uint32_t gm = row_max<4>(max_magnitude(x[i]));   // a group is 4 chunks
      const bool poison = gm >= kInfBits;
      const uint32_t sb = poison ? 0x7FC0u : f32_to_bf16(bf16_to_f32(gm) / 7.0f);
      const float s = bf16_to_f32(sb);
      const bool zero = poison || !(s > 0.f);   // codes 0
      const Divisor by(zero ? 1.0f : s);
      uint32_t u[8];
      float f[8];
      by(x[i], f);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float q = __builtin_amdgcn_fmed3f(rintf(f[t]), -8.0f, 7.0f);
        u[t] = zero ? 8u : (uint32_t)((int)q + 8);
      }
      if (pl.live && c == 0) {
        reinterpret_cast<uint16_t*>(scales)[((pl.r >> 2) * NG + g) * 4 + j] = (uint16_t)sb;
        if (poison && a.counters) atomicAdd(a.counters + 1, 1ull);
      }
      if constexpr (!V) {
        uint32_t w = 0;
#pragma unroll
        for (int t = 0; t < 8; ++t) w |= u[t] << tile16_bit(t);
        if (pl.live) *reinterpret_cast<uint32_t*>(codes + k_offset<FMT, NG>(ch, pl.r)) = w;
      } else {
        uint32_t w = 0;   // byte t: dimensions 2t (low nibble) and 2t + 1
#pragma unroll
        for (int t = 0; t < 4; ++t) w |= (u[2 * t] | (u[2 * t + 1] << 4)) << (8 * t);
        if (pl.quads) {
          *reinterpret_cast<uint32_t*>(codes + v_offset<FMT, NG>(ch, pl.r, pl.q)) = quad_transpose_bytes(w, pl.q);
        } else if (pl.live) {
#pragma unroll
          for (int t = 0; t < 4; ++t) codes[v_offset<FMT, NG>(ch, pl.r, t) + j] = (uint8_t)(w >> (8 * t));
        }
      }
    }
  }
}

// HB heads of K and V per workgroup; HB = 0: one head of K (blockIdx.z 0) or V.
template <int FMT, int NG, int HB>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(KvArgs a) {
  typedef RowSplit<NG> S;
  constexpr int D = 32 * NG;
  const Place pl = find_place<NG>(a);
  const int h0 = blockIdx.y * (HB > 0 ? HB : 1);
  if (a.counters && h0 == 0 && blockIdx.z == 0 && pl.ch == 0 && pl.slot >= 0 && !pl.live) atomicAdd(a.counters, 1ull);
  auto load = [&](u32x4 (&x)[S::CPT], const uint16_t* rows, int64_t stride, int head) {
#pragma unroll
    for (int i = 0; i < S::CPT; ++i) {
      x[i] = u32x4{0u, 0u, 0u, 0u};
      if (pl.live && head < a.kv_heads)
        x[i] = *reinterpret_cast<const u32x4*>(rows + pl.tok * stride + (int64_t)head * D + 8 * (pl.ch + S::LP * i));
    }
  };
  if constexpr (HB == 0) {
    u32x4 x[S::CPT];
    if (blockIdx.z == 0) {
      load(x, a.k, a.k_stride, h0);
      write_row<FMT, NG, false>(a, pl, x, h0);
    } else {
      load(x, a.v, a.v_stride, h0);
      write_row<FMT, NG, true>(a, pl, x, h0);
    }
  } else {
    u32x4 k[HB][S::CPT], v[HB][S::CPT];
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      load(k[h], a.k, a.k_stride, h0 + h);
      load(v[h], a.v, a.v_stride, h0 + h);
    }
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      if (h0 + h >= a.kv_heads) break;
      write_row<FMT, NG, false>(a, pl, k[h], h0 + h);
      write_row<FMT, NG, true>(a, pl, v[h], h0 + h);
    }
  }
}

// A lane's piece of a row, as it lies in the cache; where `quads` V pieces are
// those of the lane's own unit lane, still to be exchanged.
template <int FMT, int NG>
struct RowPiece {
  u32x4 w[RowSplit<NG>::CPT];   // codes: bf16 4 words, E4M3 2, Q4 1
  float s[RowSplit<NG>::CPT];
};

template <int FMT, int NG, bool V>
__device__ __forceinline__ void load_row(const KvArgs& a, const Place& pl, int head, RowPiece<FMT, NG>& o) {
  typedef KvLayout<FMT, NG> L;
  typedef RowSplit<NG> S;
  const uint8_t* block = pl.page + (int64_t)head * 2 * a.block_bytes + (V ? a.block_bytes : 0);
  const uint8_t* codes = block + (uint32_t)pl.tile * (uint32_t)L::kTileBytes;
  const uint8_t* scales = block + ((uint32_t)L::kTileBytes << a.page_shift) / kKvTile + pl.tile * L::kScaleTileBytes;
  const int j = pl.r & 3;
#pragma unroll
  for (int i = 0; i < S::CPT; ++i) {
    const int ch = pl.ch + S::LP * i, g = ch >> 2;
    o.w[i] = u32x4{0u, 0u, 0u, 0u};
    o.s[i] = 1.0f;
    if (!pl.live) continue;
    if constexpr (FMT == W4_KV_E4M3) o.s[i] = reinterpret_cast<const float*>(scales)[pl.r];
    if constexpr (FMT == W4_KV_Q4)
      o.s[i] = bf16_to_f32(reinterpret_cast<const uint16_t*>(scales)[((pl.r >> 2) * NG + g) * 4 + j]);
    if (!V || pl.quads) {
      const uint8_t* p = codes + (V ? v_offset<FMT, NG>(ch, pl.r, pl.q) : k_offset<FMT, NG>(ch, pl.r));
      if constexpr (FMT == W4_KV_BF16) {
        o.w[i] = *reinterpret_cast<const u32x4*>(p);
      } else if constexpr (FMT == W4_KV_E4M3) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p);
        o.w[i][0] = w[0];
        o.w[i][1] = w[1];
      } else {
        o.w[i][0] = *reinterpret_cast<const uint32_t*>(p);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint8_t* p = codes + v_offset<FMT, NG>(ch, pl.r, t);
        if constexpr (FMT == W4_KV_BF16) {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(p) + j;
          o.w[i][t] = h[0] | ((uint32_t)h[4] << 16);
        } else if constexpr (FMT == W4_KV_E4M3) {
          o.w[i][t >> 1] |= (p[j] | ((uint32_t)p[4 + j] << 8)) << (16 * (t & 1));
        } else {
          o.w[i][0] |= (uint32_t)p[j] << (8 * t);
        }
      }
    }
  }
}

template <int FMT, int NG, bool V, typename OUT>
__device__ __forceinline__ void store_row(const KvArgs& a, const Place& pl, int head, const RowPiece<FMT, NG>& x) {
  typedef RowSplit<NG> S;
  OUT* dst = reinterpret_cast<OUT*>(V ? a.v_out : a.k_out) + pl.tok * (V ? a.v_stride : a.k_stride) +
             (int64_t)head * (32 * NG);
#pragma unroll
  for (int i = 0; i < S::CPT; ++i) {
    u32x4 w = x.w[i];
    if (V && pl.quads) {
      if constexpr (FMT == W4_KV_BF16) {   // [b][j] -> pairs of the 4 tokens, exchanged
        w = quad_transpose(u32x4{low_halves(w[0], w[2]), high_halves(w[0], w[2]), low_halves(w[1], w[3]),
                                 high_halves(w[1], w[3])}, pl.q);
      } else if constexpr (FMT == W4_KV_E4M3) {
        const u32x2 y = quad_planes_to_pairs(u32x2{w[0], w[1]}, pl.q);
        w[0] = y[0];
        w[1] = y[1];
      } else {
        w[0] = quad_transpose_bytes(w[0], pl.q);
      }
    }
    if (!pl.live) continue;
    OUT* o = dst + 8 * (pl.ch + S::LP * i);
    if constexpr (FMT == W4_KV_BF16 && sizeof(OUT) == 2) {
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(o));
      continue;
    }
    float f[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if constexpr (FMT == W4_KV_BF16) {
        f[t] = value_of(w, t);
      } else if constexpr (FMT == W4_KV_E4M3) {
        f[t] = x.s[i] * __builtin_amdgcn_cvt_f32_fp8((int)((w[t >> 2] >> (8 * (t & 3))) & 0xFFu), 0);
      } else {
        const uint32_t u = V ? w[0] >> (4 * t) : w[0] >> tile16_bit(t);
        f[t] = x.s[i] * (float)((int)(u & 0xFu) - 8);
      }
    }
    if constexpr (sizeof(OUT) == 4) {
      __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4*>(o));
      __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f32x4*>(o + 4));
    } else {
      u32x4 y;
#pragma unroll
      for (int t = 0; t < 4; ++t) y[t] = f32_to_bf16(f[2 * t]) | (f32_to_bf16(f[2 * t + 1]) << 16);
      __builtin_nontemporal_store(y, reinterpret_cast<u32x4*>(o));
    }
  }
}

template <int FMT, int NG, int HB, typename OUT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(KvArgs a) {
  const Place pl = find_place<NG>(a);
  const int h0 = blockIdx.y * (HB > 0 ? HB : 1);
  if (a.counters && h0 == 0 && blockIdx.z == 0 && pl.ch == 0 && pl.slot >= 0 && !pl.live) atomicAdd(a.counters, 1ull);
  if constexpr (HB == 0) {
    RowPiece<FMT, NG> x;
    if (blockIdx.z == 0) {
      load_row<FMT, NG, false>(a, pl, h0, x);
      store_row<FMT, NG, false, OUT>(a, pl, h0, x);
    } else {
      load_row<FMT, NG, true>(a, pl, h0, x);
      store_row<FMT, NG, true, OUT>(a, pl, h0, x);
    }
  } else {
    RowPiece<FMT, NG> k[HB], v[HB];
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      const int head = h0 + h < a.kv_heads ? h0 + h : h0;   // past the last head: loaded again, not stored
      load_row<FMT, NG, false>(a, pl, head, k[h]);
      load_row<FMT, NG, true>(a, pl, head, v[h]);
    }
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      if (h0 + h >= a.kv_heads) break;
      store_row<FMT, NG, false, OUT>(a, pl, h0 + h, k[h]);
      store_row<FMT, NG, true, OUT>(a, pl, h0 + h, v[h]);
    }
  }
}

template <int NG>
unsigned row_blocks(const KvArgs& a) {
  return (unsigned)((a.tokens + RowSplit<NG>::ROWS - 1) / RowSplit<NG>::ROWS);
}

template <int FMT, int NG, int HB>
void launch_write(const KvArgs& a, hipStream_t stream) {
  const dim3 grid(row_blocks<NG>(a), a.kv_heads, HB > 0 ? 1 : 2);
  kv_write_kernel<FMT, NG, HB><<<grid, kThreads, 0, stream>>>(a);
}

template <int FMT, int NG, int HB>
void launch_read(const KvArgs& a, int out_dtype, hipStream_t stream) {
  constexpr int H = HB > 0 ? HB : 1;
  const dim3 grid(row_blocks<NG>(a), (a.kv_heads + H - 1) / H, HB > 0 ? 1 : 2);
  if (out_dtype == W4_OUT_F32) kv_read_kernel<FMT, NG, HB, float><<<grid, kThreads, 0, stream>>>(a);
  else kv_read_kernel<FMT, NG, HB, uint16_t><<<grid, kThreads, 0, stream>>>(a);
}

// By the call's (16 tokens x head) pieces.  Few of them: K and V to workgroups
// of their own (64 Q4 tokens of 8 x 128: write 3.3 against 4.0 us, read 3.0
// against 3.6; 2045 tokens of 4 x 256: write 5.9 against 6.5).  Many: one
// workgroup for both (write of 4096 E4M3 tokens of 8 x 128: 8.9 against 9.5
// us), and when reading for two heads (8192 tokens: 9.7 against 10.8 us; 30715
// Q4 tokens of 4 x 256: 29.1 against 30.3).
constexpr int64_t kBoth = 1024, kTwoHeads = 2048;

template <int FMT, int NG>
void launch_fmt(const KvArgs& a, bool write, int out_dtype, hipStream_t stream) {
  const int64_t wgs = (int64_t)row_blocks<NG>(a) * a.kv_heads;
  if (write) {
    if (wgs >= kBoth) launch_write<FMT, NG, 1>(a, stream);
    else launch_write<FMT, NG, 0>(a, stream);
  } else if (wgs >= kTwoHeads && a.kv_heads > 1) {
    launch_read<FMT, NG, 2>(a, out_dtype, stream);
  } else if (wgs >= kBoth) {
    launch_read<FMT, NG, 1>(a, out_dtype, stream);
  } else {
    launch_read<FMT, NG, 0>(a, out_dtype, stream);
  }
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
