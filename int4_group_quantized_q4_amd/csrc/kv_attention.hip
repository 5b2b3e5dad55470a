// Attention of one new token per sequence over the paged key-value cache.
//
//   s_t = scale * q . k_t,  out = sum_t softmax(s)_t v_t,  lse = log sum_t e^(s_t)
//
// over the positions [max(0, len - window), len) of a sequence, for the G =
// heads / kv_heads query heads that share a kv head.  One pass over the cache
// with the running maximum and sum of the softmax.
//
// Bound by the cache's bytes: a token's K and V row of a head are read once
// for 16 query heads (more of them read it again: bf16 32 x 32768 of 2 x 128
// 170 us with 16 heads a kv head, 330 with 32).  bf16 8 x 32768 tokens of 8 x
// 128: 161 us, 6.7 TB/s; E4M3 48 ragged sequences up to 8000 of 8 x 128: 54 us,
// 5.1 TB/s; Q4 16 x 32768 of 8 x 128, 8 heads a kv head: 129 us, 4.7 TB/s (Q4 by
// the vector instructions that unpack, scale and split, and the clock they
// leave; 32 x 16384 of 8 x 64: 76 us, 4.0 TB/s).
//
// Work split: grid (kv head x tile of 16 query heads, items), an item being a
// run of a sequence's positions; a workgroup of 4 waves takes one, and a wave
// 32 tokens at a time (two tiles of the cache), with its own running maximum,
// sum and output.  The waves are joined through LDS, the items of a sequence
// by a second kernel.  Few short sequences go to workgroups of 8 waves, whole.
//
// Matrix layouts (16x16x32 bf16, lane = 16c + n): the scores are formed as
// S^T = K . Q^T with a tile's 16 tokens as rows, so lane (c, n) holds the
// scores of head n for tokens 4c .. 4c+3 of both tiles.  Those 8 values are
// the lane's B operand of O^T = V^T . P^T when the 32 tokens are numbered (c,
// tile, j), and the cache keeps V so that one lane's load holds those tokens
// of dimension 32g + 2n + b: no value crosses lanes between the two products.
//
// Q4's scales differ from group to group, and applying them is what its
// vector instructions would go into.  With at most 8 (4) heads the 16 columns
// hold R = 2 (4) replicas of each head, and replica r does the scale
// arithmetic of the r-th part of the groups: its q is zero in the others, its
// part of the scores is summed over the replicas by lane rotations, and of
// the second product a group's rows count in its own replica's columns only.
//
// Precision: q and the codes are exact in bf16 and all sums are fp32 (Q4: with
// the codes as 8 + q, which an fp32 sum rounds about as much as the group's
// largest values, whose codes are 7 and -7 or -8, make it round anyway).  The
// probabilities (times the V scales) enter the second product as three bf16
// terms that hold their 24 bits.

#include <type_traits>

#include "common.h"
#include "decode.h"
#include "kv_layout.h"
#include "w4a16.h"

namespace w4 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Least waves per SIMD that the register allocator keeps (none spills at these).
constexpr int waves_per_simd(int fmt, int ng) { return ng == 2 ? 4 : ng == 4 && fmt != W4_KV_BF16 ? 3 : 2; }

constexpr int kWaves = 4;
constexpr int kWideWaves = 8;       // of a workgroup that takes a short row alone
constexpr int kChunk = 32;          // tokens per wave step
constexpr float kSlack = 8.0f;       // of the softmax's running reference above the maximum, in powers of two
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

// 4 E4M3 codes -> 4 bf16 (two words), exact
__device__ __forceinline__ u32x2 e4m3_to_bf16(uint32_t w) {
  u32x2 o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
  return o;
}

// Q4: four codes u = q + 8, one in each byte -> bf16 u, exact: as an E4M3 code
// a byte up to 15 stands for u 2^-9 (the subnormals and the first binade, which
// have one step).  As 136 + q, by byte permutes, sums were rounded 17 times as
// much, for 125 us instead of 129 (16 x 32768 tokens of 8 x 128).
__device__ __forceinline__ u32x2 q4_to_bf16(uint32_t w) {
  u32x2 o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, false));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, true));
  return o;
}
// A K word's 8 codes, in the order of its bytes: dimensions 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ u32x4 q4_word_to_bf16(uint32_t w) {
  const u32x2 lo = q4_to_bf16(w & 0x0F0F0F0Fu), hi = q4_to_bf16((w >> 4) & 0x0F0F0F0Fu);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}
// q's 8 dimensions in that order.
__device__ __forceinline__ u32x4 q4_word_order(u32x4 q) {
  return u32x4{__builtin_amdgcn_perm(q[2], q[0], 0x05040100u), __builtin_amdgcn_perm(q[2], q[0], 0x07060302u),
               __builtin_amdgcn_perm(q[3], q[1], 0x05040100u), __builtin_amdgcn_perm(q[3], q[1], 0x07060302u)};
}
constexpr uint32_t kNeg8Pair = 0xC100C100u;   // bf16 -8

__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// 8 fp32 values -> three bf16 terms each, whose sum is the value: 8 of its 24
// bits at a time, by truncation (the differences are exact).  Two terms (16
// bits) took 112 us instead of 125 for Q4 16 x 32768 tokens of 8 x 128, and as
// long as three where memory bounds the call (bf16, E4M3).
__device__ __forceinline__ void split_bf16(const float p[8], u32x4& hi, u32x4& mid, u32x4& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[2][3];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float v = p[2 * i + k];
      const float r = v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
      w[k][0] = __float_as_uint(v);
      w[k][1] = __float_as_uint(r);
      w[k][2] = __float_as_uint(r - __uint_as_float(__float_as_uint(r) & 0xFFFF0000u));
    }
    hi[i] = __builtin_amdgcn_perm(w[1][0], w[0][0], 0x07060302u);   // the upper halves
    mid[i] = __builtin_amdgcn_perm(w[1][1], w[0][1], 0x07060302u);
    lo[i] = __builtin_amdgcn_perm(w[1][2], w[0][2], 0x07060302u);
  }
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return mfma16x16x32(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c);
}

// over the four lanes of one column n
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// The value N columns on (of 16).
template <int N>
__device__ __forceinline__ float rotated(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + N, 0xF, 0xF, true));
}

// 1 / l and the log of the sum of a row: l is 0 for an empty one; NaN passes on.
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l; }
__device__ __forceinline__ float log_sum(float m, float l) {
  return l > 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : l == 0.f ? -INFINITY : l;
}

// The positions a sequence attends to, and their 32-token chunks.
struct Span {
  int n, lo;          // positions [lo, n); all positions fit 31 bits
  int first, chunks;  // chunk range
};

__device__ __forceinline__ Span span_of(const AttnArgs& a, int len) {
  Span s;
  const int most = (int)a.table_width << a.page_shift;
  s.n = len < 0 ? 0 : len > most ? most : len;
  s.lo = a.window > 0 && s.n > a.window ? s.n - a.window : 0;
  s.first = s.lo / kChunk;
  s.chunks = (int)(((unsigned)s.n + kChunk - 1) / kChunk) - s.first;
  return s;
}

// Inclusive prefix sum over the wave.
__device__ __forceinline__ int wave_prefix(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);    // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast 15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast 31 into rows 2 and 3
  return v;
}

// Work items of a call whose positions are split: a fair share is the batch's
// chunks divided by `shares`, and a sequence is cut into equal items of about
// one share (at most a quarter more, as an item much smaller than the others
// costs its start and end; one item for an empty sequence), so that long and
// short sequences get workgroups by their length.  The lengths are on the
// device, so every wave counts the items for itself.
struct Item {
  int seq, index;     // sequence of the item and its place in it
  int base, live;     // the sequence's first item and their number
  int len;
  bool found;
};

__device__ __forceinline__ Item find_item(const AttnArgs& a, int want) {
  const int lane = threadIdx.x & 63;
  const int seqs = (int)a.seqs;
  const bool small = (a.table_width << a.page_shift) < ((int64_t)1 << 29);   // 64 chunk counts fit 31 bits
  int64_t total = a.shares - 1;
  int len = 0, chunks = 0;
  for (int b = 0; b < seqs; b += 64) {
    const int l = b + lane < seqs ? a.lens[b + lane] : 0;
    const int ch = span_of(a, l).chunks;
    if (b == 0) {
      len = l;
      chunks = ch;
    }
    if (small) {
      total += __builtin_amdgcn_readlane(wave_prefix(ch), 63);
    } else {
      const int lo = __builtin_amdgcn_readlane(wave_prefix(ch & 0xFFFF), 63);
      const int hi = __builtin_amdgcn_readlane(wave_prefix(ch >> 16), 63);
      total += ((int64_t)hi << 16) + lo;
    }
  }
  unsigned per = total < ((int64_t)1 << 31) ? (unsigned)total / (unsigned)a.shares : (unsigned)(total / a.shares);
  if (per < kWaves) per = kWaves;
  Item it{};
  for (int b = 0; b < seqs; b += 64) {
    if (b > 0) {
      len = b + lane < seqs ? a.lens[b + lane] : 0;
      chunks = span_of(a, len).chunks;
    }
    // ceil(chunks / per - 1/4), at least 1
    int cnt = (int)((4u * (unsigned)chunks + 3u * per - 1u) / (4u * per));
    if (cnt == 0) cnt = 1;
    if (b + lane >= seqs) cnt = 0;
    const int upto = wave_prefix(cnt);
    const uint64_t hit = __ballot(it.base + upto > want);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      it.seq = b + l;
      it.live = __builtin_amdgcn_readlane(cnt, l);
      it.len = __builtin_amdgcn_readlane(len, l);
      it.base += __builtin_amdgcn_readlane(upto, l) - it.live;
      it.index = want - it.base;
      it.found = true;
      return it;
    }
    it.base += __builtin_amdgcn_readlane(upto, 63);
  }
  return it;
}

template <int FMT, int NG, int R, int W>
__global__ void __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(waves_per_simd(FMT, NG))))
kv_attention_kernel(AttnArgs a) {
  typedef KvLayout<FMT, NG> L;
  constexpr int BD = NG < 4 ? 32 * NG : 128;          // dimensions joined at a time
  constexpr int HPR = 16 / R;                         // heads per replica
  constexpr int GR = NG / R;                          // groups per replica
  __shared__ float s_o[W][16][BD + 4];
  __shared__ float s_m[W][16], s_l[W][16];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, c = lane >> 4;
  const int hl = n16 % HPR, rep = n16 / HPR;          // this column's head and replica
  // heads before items: the workgroups go round the XCDs one by one
  const int hrow = blockIdx.x;
  const int head = (int)((unsigned)hrow / (unsigned)a.head_tiles), ht = hrow - head * a.head_tiles;
  int seq = blockIdx.y, index = 0, live = 1, len;
  if (a.shares > 0) {
    const Item it = find_item(a, blockIdx.y);
    if (!it.found) return;
    seq = it.seq;
    index = it.index;
    live = it.live;
    len = it.len;
    if (hrow == 0 && index == 0 && threadIdx.x == 0) a.part_plan[seq] = int2{it.base, live};   // for the join
  } else {
    len = a.lens[seq];
  }
  // the same in every lane: kept in scalar registers
  seq = __builtin_amdgcn_readfirstlane(seq);
  index = __builtin_amdgcn_readfirstlane(index);
  live = __builtin_amdgcn_readfirstlane(live);
  len = __builtin_amdgcn_readfirstlane(len);
  const int G = (int)((unsigned)a.heads / (unsigned)a.kv_heads);
  const int live_heads = G - 16 * ht < 16 ? G - 16 * ht : 16;
  const int h0 = head * G + 16 * ht;     // first query head
  const int32_t* table = a.table + (int64_t)seq * a.table_width;
  const int width = (int)a.table_width;
  const Span sp = span_of(a, len);
  if (a.counters && index == 0 && hrow == 0) {  // table entries outside the cache, once per entry
    const int p1 = (int)(((unsigned)sp.n + (1u << a.page_shift) - 1) >> a.page_shift);
    for (int p = (sp.lo >> a.page_shift) + (int)threadIdx.x; p < p1; p += 64 * W) {
      const int id = table[p];
      if (id < 0 || id >= a.n_pages) atomicAdd(a.counters, 1ull);
    }
  }

  f32x4 acc[NG][2];
  f32x4 vbias[FMT == W4_KV_Q4 ? GR : 1];   // Q4: -8 times the replica's sum of P . scale
  const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < NG; ++g) acc[g][0] = acc[g][1] = zero4;
#pragma unroll
  for (int i = 0; i < (FMT == W4_KV_Q4 ? GR : 1); ++i) vbias[i] = zero4;
  float m_run = -INFINITY, l_run = 0.f;    // l_run: this lane's tokens only
  // The scores' scale enters with the exponent, where it has to be positive for
  // the maximum: a negative one turned q round above, 0 is applied at once.
  const float scale2 = a.scale == 0.f ? 1.0f : __builtin_fabsf(a.scale) * kLog2e;

  const int size = (int)((unsigned)sp.chunks / (unsigned)live), rest = sp.chunks - size * live;
  const int begin = sp.first + index * size + (index < rest ? index : rest);
  const int end = begin + size + (index < rest ? 1 : 0);
  const int tile_shift = a.page_shift - 4;
  const uint32_t scale_off = ((uint32_t)L::kTileBytes << a.page_shift) / kKvTile;

  // The sequence's page ids, 64 table entries at a time, one per lane: a
  // chunk's ids are lane reads, with no load in front of the cache's loads.
  int ids0 = 0;
  int ids = -1;
  auto fill_ids = [&](int first) {
    ids0 = first;
    ids = -1;
    if (first + lane < width) {
      const int id = table[first + lane];
      if (id >= 0 && id < a.n_pages) ids = id;
    }
  };
  // The table first, then q, then K and V, and only then arithmetic on q (Q4 1 x
  // 1000 tokens of 8 x 128 9.1 -> 8.7 us in a graph, bf16 24 x 1000 of 4 x 128
  // 16.7 -> 15.1).
  int ch = begin + wv;
  if (ch < end) fill_ids((2 * ch) >> tile_shift);

  // q of the column's head: dimensions 32g + 8c .. of the replica's groups
  u32x4 q[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    q[g] = u32x4{0u, 0u, 0u, 0u};
    if (hl < live_heads && rep == g / GR) {
      const uint16_t* row = a.q + (int64_t)seq * a.q_stride + (int64_t)(h0 + hl) * L::D;
      q[g] = *reinterpret_cast<const u32x4*>(row + 32 * g + 8 * c);
    }
  }
  float kbias[GR];   // Q4, set once the first loads are on their way

  // One chunk's K and V (codes and scales of its two tiles), each unit loaded
  // again as soon as its registers are free.  Apart (head_dim 64 and 128): K
  // for the next chunk goes out after this chunk's scores, V after its
  // products, so one of the two is always on its way.  Shared (head_dim 256,
  // where two sets of registers would leave one wave per SIMD): K and V take
  // turns in one set, V of this chunk going out unit by unit behind the
  // scores, K of the next behind the products.
  constexpr bool SHARED = NG == 8;
  constexpr int NS = FMT == W4_KV_BF16 ? 0 : FMT == W4_KV_E4M3 ? 1 : (GR + 1) / 2;   // 16-byte scale loads per tile
  constexpr int NS1 = NS > 0 ? NS : 1;
  u32x4 kr[2][L::NU], ksr[2][NS1];
  u32x4 v_own[SHARED ? 1 : 2][SHARED ? 1 : L::NU], vs_own[SHARED ? 1 : 2][SHARED ? 1 : NS1];
  auto& vr = [&]() -> auto& { if constexpr (SHARED) return kr; else return v_own; }();
  auto& vsr = [&]() -> auto& { if constexpr (SHARED) return ksr; else return vs_own; }();
  const uint8_t* next_p[2];   // page and head block of the tiles that are loaded
  int next_tip[2];            // their place in the page
  bool good[2], next_good[2];
  // Loads take a uniform base and a 32-bit lane offset; hidden from the
  // optimizer here, which would widen it outside the loop and add in vector
  // registers.
  auto lane_offset = [](uint32_t off) {
    asm volatile("" : "+v"(off));
    return off;
  };
  auto load_unit = [&](bool v, int t, int u, u32x4& r) {
    const uint8_t* p = next_p[t] + (v ? a.block_bytes : 0) + (uint32_t)next_tip[t] * (uint32_t)L::kTileBytes;
    p += u * 64 * L::kUnitBytes;
    const uint32_t off = lane_offset((uint32_t)lane * L::kUnitBytes);
    if constexpr (L::kUnitBytes == 16) {
      r = load16(p + off);
    } else {
      const u32x2 h = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + off));
      r = u32x4{h[0], h[1], 0u, 0u};
    }
  };
  // scales of tokens 4c .. 4c+3: fp32 [j] (E4M3), bf16 [the replica's g][j] (Q4)
  auto load_scales = [&](bool v, u32x4 (&r)[2][NS1]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* p = next_p[t] + (v ? a.block_bytes : 0) + scale_off +
                         (uint32_t)next_tip[t] * (uint32_t)L::kScaleTileBytes;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if constexpr (FMT == W4_KV_Q4 && GR == 1) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(p + lane_offset((uint32_t)(8 * (c * NG + rep))));
          r[t][0] = u32x4{w[0], w[1], 0u, 0u};
        } else {
          const uint32_t at = FMT == W4_KV_Q4 ? 8 * (c * NG + rep * GR) : 16 * c;
          r[t][i] = *reinterpret_cast<const u32x4*>(p + 16 * i + lane_offset(at));
        }
      }
    }
  };
  // The places of a chunk's tiles; a tile past the table or in a page outside
  // the cache reads page 0 and is masked as a whole.
  auto find_tiles = [&](int ch) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int pi = (2 * ch + t) >> tile_shift;
      if (pi - ids0 >= 64) fill_ids(pi);
      const int id = __builtin_amdgcn_readlane(ids, pi - ids0);
      next_good[t] = id >= 0;
      next_p[t] = a.cache + (int64_t)(id >= 0 ? id : 0) * a.page_bytes + (int64_t)head * 2 * a.block_bytes;
      next_tip[t] = (2 * ch + t) & ((1 << tile_shift) - 1);
    }
  };
  auto load_k = [&](int ch) {
    find_tiles(ch);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int u = 0; u < L::NU; ++u) load_unit(false, t, u, kr[t][u]);
    load_scales(false, ksr);
  };
  auto load_v = [&]() {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int u = 0; u < L::NU; ++u) load_unit(true, t, u, vr[t][u]);
    load_scales(true, vsr);
  };
  // scale of token j (E4M3), or of token j in the replica's group i (Q4)
  auto scale_of = [&](const u32x4 (&sr)[NS1], int i, int j) {
    if constexpr (FMT == W4_KV_E4M3) return __uint_as_float(sr[0][j]);
    const uint32_t w = sr[NS > 0 ? i >> 1 : 0][2 * (i & 1) + (j >> 1)];
    return (j & 1) ? __uint_as_float(w & 0xFFFF0000u) : bf16_to_f32(w & 0xFFFFu);
  };

  // Q4: takes the codes' +8 off the outputs.  Every 8 chunks: left to the end,
  // the sums would grow to 8 times those of the probabilities, and lose that
  // much of their 24 bits where long flat attention averages the values out.
  auto take_bias = [&]() {
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[g][b] += vbias[g % GR];
#pragma unroll
    for (int i = 0; i < GR; ++i) vbias[i] = zero4;
  };

  // whether group g is the last of its unit in the order (i, r), g = r GR + i
  auto unit_done = [](int g) {
    bool last = true;
    for (int h = g / L::U * L::U; h < (g / L::U + 1) * L::U; ++h)
      if (h % GR * R + h / GR > g % GR * R + g / GR) last = false;
    return last;
  };

  // One chunk, and the loads of the wave's next one (loading the last chunk
  // again instead of a step of its own for it: E4M3 48 ragged sequences of 8 x
  // 128 57 against 53 us, bf16 64 x 1024 46.6 against 43.0).
  auto step = [&](int ch, auto last) {
    constexpr bool LAST = decltype(last)::value;
    good[0] = next_good[0];
    good[1] = next_good[1];
    float p[8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f32x4 s4 = zero4;
      // groups in the order of their scale arithmetic: a replica's i-th for all replicas
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        float kb = kbias[i];
        // four registers each over the loop are too many for more than two of them
        if constexpr (GR > 2) asm volatile("" : "+v"(kb));
        f32x4 d = {kb, kb, kb, kb};
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int g = r * GR + i, u = g / L::U, part = g % L::U;
          if constexpr (NG == 8) __builtin_amdgcn_sched_barrier(0);
          if constexpr (FMT == W4_KV_BF16) {
            s4 = mfma(kr[t][u], q[g], s4);
          } else if constexpr (FMT == W4_KV_E4M3) {
            const u32x2 a0 = e4m3_to_bf16(kr[t][u][2 * part]), a1 = e4m3_to_bf16(kr[t][u][2 * part + 1]);
            s4 = mfma(u32x4{a0[0], a0[1], a1[0], a1[1]}, q[g], s4);
          } else {
            // a column gathers its replica's groups only (its q is zero in the others)
            d = mfma(q4_word_to_bf16(kr[t][u][part]), q[g], d);
          }
          if (SHARED && unit_done(g)) {
            __builtin_amdgcn_sched_barrier(0);
            load_unit(true, t, u, vr[t][u]);
          }
        }
        if constexpr (FMT == W4_KV_Q4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) s4[j] = fmaf(scale_of(ksr[t], i, j), d[j], s4[j]);
        }
      }
      // Q4: over the replicas; in this order every replica gets the same bits
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (R >= 2) s4[j] += rotated<8>(s4[j]);
        if constexpr (R >= 4) s4[j] += rotated<4>(s4[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) p[4 * t + j] = FMT == W4_KV_E4M3 ? s4[j] * scale_of(ksr[t], 0, j) : s4[j];
    }
    if (a.scale == 0.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] *= 0.f;
    }
    __builtin_amdgcn_sched_barrier(0);   // not before the scores: K's registers are reused
    if constexpr (SHARED) {
      load_scales(true, vsr);
      if constexpr (!LAST) find_tiles(ch + W);
    } else if constexpr (!LAST) {
      load_k(ch + W);
    }

    // Positions outside the span or in pages outside the cache have no score,
    // and what their V rows hold (anything) is cleared, since 0 * NaN is NaN.
    if (ch * kChunk < sp.lo || ch * kChunk > sp.n - kChunk || !good[0] || !good[1]) {
      int rel = ch * kChunk + 4 * c;
      asm volatile("" : "+v"(rel));   // keeps the positions' arithmetic inside this branch
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t keep = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pos = rel + 16 * t + j;
          const bool in = good[t] && pos >= sp.lo && pos < sp.n;
          if (!in) p[4 * t + j] = -INFINITY;
          keep |= in ? 0xFFu << (8 * j) : 0u;
        }
        // byte masks widened to the words that hold (tokens 0 and 1) and (2 and 3)
        const uint32_t k01 = ((keep & 0xFFu) | ((keep & 0xFF00u) << 8)) * 0x101u;
        const uint32_t k23 = (((keep >> 16) & 0xFFu) | ((keep >> 24) << 16)) * 0x101u;
        // an operand's lane (c, m) holds tokens 4c + j, as the scores' lane (c, n) does
#pragma unroll
        for (int u = 0; u < L::NU; ++u) {
          if constexpr (FMT == W4_KV_BF16) {
            vr[t][u][0] &= k01;
            vr[t][u][1] &= k23;
            vr[t][u][2] &= k01;
            vr[t][u][3] &= k23;
          } else if constexpr (FMT == W4_KV_E4M3) {
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[t][u][i] &= keep;
          }
        }
        if constexpr (FMT == W4_KV_E4M3) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!((keep >> (8 * j)) & 1u)) vsr[t][0][j] = 0u;
        } else if constexpr (FMT == W4_KV_Q4) {
#pragma unroll
          for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) vsr[t][i][w] &= (w & 1) ? k23 : k01;
        }
      }
    }

    // Softmax against a running reference: any reference gives the same
    // result, so it is set 2^kSlack above the maximum and follows only when the
    // maximum has passed it: the outputs are rarely rescaled, and no p is over
    // 1, so the sums hold no more than the values' own.
    float top = p[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, p[i]);
    top = column_max(top) * scale2;
    if (__any(top > m_run)) {
      const float m_new = fmaxf(m_run, top + kSlack);
      const float alpha = m_new == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m_run - m_new);
      m_run = m_new;
      l_run *= alpha;
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[g][b] *= alpha;
      if constexpr (FMT == W4_KV_Q4) {
#pragma unroll
        for (int i = 0; i < GR; ++i) vbias[i] *= alpha;
      }
    }
    const float m_use = m_run == -INFINITY ? 0.f : m_run;   // nothing yet: every p is 0
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[i], scale2, -m_use));
      sum += p[i];
    }
    l_run += sum;

    // O^T += V^T . P^T (Q4: P times the scales of the replicas' i-th groups)
    u32x4 ph, pm, pl;
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      if (FMT == W4_KV_Q4 || i == 0) {
        float ps[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) ps[k] = FMT == W4_KV_BF16 ? p[k] : p[k] * scale_of(vsr[k >> 2], i, k & 3);
        split_bf16(ps, ph, pm, pl);
      }
      if constexpr (FMT == W4_KV_Q4) {
        const u32x4 bias = {kNeg8Pair, kNeg8Pair, kNeg8Pair, kNeg8Pair};
        vbias[i] = mfma(bias, ph, vbias[i]);
        vbias[i] = mfma(bias, pm, vbias[i]);
        vbias[i] = mfma(bias, pl, vbias[i]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int g = r * GR + i, u = g / L::U, part = g % L::U;
        if constexpr (NG == 8) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          u32x4 av;
          if constexpr (FMT == W4_KV_BF16) {
            av = u32x4{vr[0][u][2 * b], vr[0][u][2 * b + 1], vr[1][u][2 * b], vr[1][u][2 * b + 1]};
          } else if constexpr (FMT == W4_KV_E4M3) {
            const u32x2 a0 = e4m3_to_bf16(vr[0][u][2 * part + b]), a1 = e4m3_to_bf16(vr[1][u][2 * part + b]);
            av = u32x4{a0[0], a0[1], a1[0], a1[1]};
          } else {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              // byte j: token j's code of dimension 2m (low nibble), 2m + 1 (high)
              const u32x2 w = q4_to_bf16((b ? vr[t][u][part] >> 4 : vr[t][u][part]) & 0x0F0F0F0Fu);
              av[2 * t] = w[0];
              av[2 * t + 1] = w[1];
            }
          }
          acc[g][b] = mfma(av, ph, acc[g][b]);
          acc[g][b] = mfma(av, pm, acc[g][b]);
          acc[g][b] = mfma(av, pl, acc[g][b]);
        }
        if (SHARED && !LAST && unit_done(g)) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int t = 0; t < 2; ++t) load_unit(false, t, u, kr[t][u]);
        }
      }
    }
    if constexpr (!LAST) {
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (SHARED) load_scales(false, ksr);
      else load_v();
    }
  };

  if (ch < end) {
    load_k(ch);
    // in this order, as in the loop: loads complete in order, and waiting for K
    // must not mean waiting for V
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!SHARED) load_v();
    __builtin_amdgcn_sched_barrier(0);
    if (a.scale < 0.f) {
#pragma unroll
      for (int g = 0; g < NG; ++g) q[g] ^= 0x80008000u;
    }
    // Q4 codes enter as 8 + q: -8 times q's sum over each group cancels that
    if constexpr (FMT == W4_KV_Q4) {
#pragma unroll
      for (int g = 0; g < NG; ++g) q[g] = q4_word_order(q[g]);
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)     // all but the replica's own are zero
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t w = q[r * GR + i][k];
            t += bf16_to_f32(w & 0xFFFFu) + __uint_as_float(w & 0xFFFF0000u);
          }
        kbias[i] = -8.0f * column_sum(t);
      }
    }
    for (int i = 1; ch + W < end; ch += W, ++i) {
      step(ch, std::false_type());
      if (FMT == W4_KV_Q4 && (i & 7) == 0) take_bias();
    }
    step(ch, std::true_type());
  }
  if constexpr (FMT == W4_KV_Q4) take_bias();

  // Join the waves: lane (c, n) holds, for group g, dimensions 32g + 8c + 2i + b.
  const float l_col = column_sum(l_run);
  if (c == 0) {
    s_m[wv][n16] = m_run;
    s_l[wv][n16] = l_col;
  }
  __syncthreads();
  float m_all = -INFINITY;
#pragma unroll
  for (int w = 0; w < W; ++w) m_all = fmaxf(m_all, s_m[w][n16]);
  const float mine = m_run == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m_run - m_all);
  constexpr int ROUNDS = 32 * NG / BD;
#pragma unroll
  for (int rd = 0; rd < ROUNDS; ++rd) {
    if (rd) __syncthreads();
#pragma unroll
    for (int g = 0; g < BD / 32; ++g) {
      if (R > 1 && rep != (rd * (BD / 32) + g) / GR) continue;   // another replica's
      float* o = &s_o[wv][hl][32 * g + 8 * c];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = acc[rd * (BD / 32) + g][0][i] * mine;
        o[2 * i + 1] = acc[rd * (BD / 32) + g][1][i] * mine;
      }
    }
    __syncthreads();
    // thread -> 4 dimensions of one head
    for (int e = threadIdx.x; e < live_heads * (BD / 4); e += 64 * W) {
      const int h = e / (BD / 4), d = 4 * (e % (BD / 4));
      float mx = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[w][h]);
      f32x4 o = zero4;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        // a wave without a score has l = 0 (or NaN, which passes on)
        l += s_m[w][h] == -INFINITY ? s_l[w][h] : s_l[w][h] * __builtin_amdgcn_exp2f(s_m[w][h] - mx);
        o += *reinterpret_cast<const f32x4*>(&s_o[w][h][d]);
      }
      const int64_t row = (int64_t)seq * a.heads + h0 + h;
      const int dim = rd * BD + d;
      if (live == 1) {
        const float inv = inverse_sum(l);
        u32x2 w2 = {pk_bf16(o[0] * inv, o[1] * inv), pk_bf16(o[2] * inv, o[3] * inv)};
        *reinterpret_cast<u32x2*>(a.out + row * L::D + dim) = w2;
        if (a.lse && dim == 0) a.lse[row] = log_sum(mx, l);
      } else {
        const int64_t pr = (int64_t)blockIdx.y * a.heads + h0 + h;
        *reinterpret_cast<f32x4*>(a.part_o + pr * L::D + dim) = o;
        if (dim == 0) {
          a.part_ml[2 * pr] = mx;
          a.part_ml[2 * pr + 1] = l;
        }
      }
    }
  }
}

// Joins the splits of one (sequence, query head): D/4 threads take 4 dimensions
// each of one split, the workgroup's 1024/D such groups take splits in turn
// and are added in LDS, in group order (fp32; the order depends on the split
// count alone).  Bound by latency: lengths, then maxima and sums, then the
// outputs, each level's loads in flight together.
template <int NG>
__global__ void __launch_bounds__(256) kv_join_kernel(AttnArgs a) {
  constexpr int D = 32 * NG, TG = D / 4, GROUPS = 256 / TG;
  __shared__ f32x4 s_o[GROUPS][TG];
  const int lane = threadIdx.x & 63;
  const int2 plan = a.part_plan[blockIdx.y];
  const int live = plan.y;
  if (live <= 1) return;   // the attention kernel wrote the output
  const int64_t row = (int64_t)blockIdx.y * a.heads + blockIdx.x;
  const int64_t first = (int64_t)plan.x * a.heads + blockIdx.x;    // the row's first partial result
  const int pitch = 2 * a.heads;
  const float* ml = a.part_ml + 2 * first;
  // every wave reduces all (m, l) pairs
  float mx = -INFINITY;
  for (int s = lane; s < live; s += 64) mx = fmaxf(mx, ml[(int64_t)s * pitch]);
  mx = wave_max_all(mx);
  // an item without a score has l = 0 and o = 0 (or NaN, which passes on)
  auto weight = [&](float m) { return m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mx); };
  float l = 0.f;
  for (int s = lane; s < live; s += 64) l += ml[(int64_t)s * pitch + 1] * weight(ml[(int64_t)s * pitch]);
  l = wave_sum_all(l);

  const int grp = threadIdx.x / TG, d = threadIdx.x % TG;
  const f32x4* po = reinterpret_cast<const f32x4*>(a.part_o + first * D) + d;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int s = grp; s < live; s += 4 * GROUPS) {
    f32x4 v[4];
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = s + i * GROUPS;
      v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      w[i] = 0.f;
      if (k < live) {
        v[i] = po[(int64_t)k * a.heads * TG];
        w[i] = weight(ml[(int64_t)k * pitch]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o += v[i] * w[i];
  }
  s_o[grp][d] = o;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int i = 1; i < GROUPS; ++i) o += s_o[i][d];
  const float inv = inverse_sum(l);
  *reinterpret_cast<u32x2*>(a.out + row * D + 4 * d) =
      u32x2{pk_bf16(o[0] * inv, o[1] * inv), pk_bf16(o[2] * inv, o[3] * inv)};
  if (a.lse && d == 0) a.lse[row] = log_sum(mx, l);
}

// Replicas of the heads, Q4 only: as many as fit.  16 x 32768 tokens of 8 x
// 128, 8 heads a kv head: 156 us with R = 1, 129 with 2; 4 heads: 152, 124, and
// 113 with 4; of 4 x 256, 4 heads: 160, 133, 118; 32 x 16384 of 8 x 64: 88, 76.
template <int FMT, int NG, int W>
void launch_fmt(const AttnArgs& a, dim3 grid, hipStream_t stream) {
  constexpr int MOST = FMT != W4_KV_Q4 ? 1 : NG < 4 ? 2 : 4, HALF = MOST < 2 ? 1 : 2;
  const int G = a.heads / a.kv_heads;
  if (G <= 16 / MOST) kv_attention_kernel<FMT, NG, MOST, W><<<grid, 64 * W, 0, stream>>>(a);
  else if (G <= 16 / HALF) kv_attention_kernel<FMT, NG, HALF, W><<<grid, 64 * W, 0, stream>>>(a);
  else kv_attention_kernel<FMT, NG, 1, W><<<grid, 64 * W, 0, stream>>>(a);
}

template <int FMT, int W>
void launch_dim(const AttnArgs& a, dim3 grid, hipStream_t stream) {
  if (a.head_dim == 64) launch_fmt<FMT, 2, W>(a, grid, stream);
  else if (a.head_dim == 128) launch_fmt<FMT, 4, W>(a, grid, stream);
  else launch_fmt<FMT, 8, W>(a, grid, stream);
}

template <int FMT>
void launch_waves(const AttnArgs& a, bool wide, dim3 grid, hipStream_t stream) {
  if (wide) launch_dim<FMT, kWideWaves>(a, grid, stream);
  else launch_dim<FMT, kWaves>(a, grid, stream);
}

int64_t head_tiles_of(int32_t heads, int32_t kv_heads) { return (heads / kv_heads + 15) / 16; }

// How a call's positions are split.  The workgroups aimed at are those that
// keep the memory busy: fewer and longer ones lose less in starts, ends and
// partial results.  Measured (us; 256, 512, 768, 1024 workgroups): bf16 8 x
// 32768 tokens of 8 x 128: 163, 169, 171, 168; bf16 32 x 8192 of 8 x 64: 85,
// 90, 89, 89; bf16 16 x 8192 of 4 x 256: 89, 90, 92, 92; E4M3 32 x 32768
// ragged of 8 x 128: 154, 143, 133, 129; E4M3 16 x 16384 of 8 x 128: 88, 91,
// 91, 91; E4M3 16 x 16384 of 4 x 256: 90, 91, 100, 93; Q4 16 x 32768 of 8 x
// 128: 162, 135, 128, 128; Q4 32 x 16384 of 8 x 64: 117, 86, 80, 77; Q4 16 x
// 32768 of 4 x 256: 165, 117, 128, 122.
int64_t target_of(int32_t format, int32_t head_dim) {
  if (format == W4_KV_BF16) return 256;
  if (format == W4_KV_E4M3) return head_dim == 256 ? 256 : 768;
  return head_dim == 64 ? 1024 : head_dim == 128 ? 768 : 512;
}
constexpr int64_t kMostTarget = 1024;

struct Plan {
  int shares;     // 0: one workgroup per sequence and head row
  bool wide;      // of 8 waves
  int64_t items;  // at most
};

// `tokens`: the most a sequence attends to.  A call with enough sequences and
// head rows is split too where a long sequence among short ones would outlast
// the others (over kUnsplit tokens), unless counting the items takes too long.
constexpr int64_t kUnsplit = 4096, kMostCounted = 256;

// With too few rows to fill the card, splitting a short row costs more (a
// second launch and its start) than one workgroup of 8 waves takes for it.  In
// tokens x dimensions (us in a graph, split against wide): Q4 1 x 500 tokens of
// 8 x 128: 8.9, 8.1; 1 x 1000: 8.9, 11.1; 1 x 250 of 4 x 256: 10.3, 9.2; 1 x
// 500: 10.4, 11.8; with more rows up to twice as far (12 x 1000 of 8 x 128:
// 12.1, 11.5; bf16 17.0, 15.1; Q4 12 x 2000: 14.7, 17.8).
constexpr int64_t kWide = 512 * 128, kWideManyRows = 2 * kWide, kManyRows = 64;

Plan plan_of(int64_t target, int64_t seqs, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t tokens) {
  const int64_t hrows = kv_heads * head_tiles_of(heads, kv_heads);
  const int64_t most = (tokens + kWaves * kChunk - 1) / (kWaves * kChunk);   // items a sequence can have
  const bool enough = seqs * hrows * 3 >= target * 2;
  if (most <= 1 || (enough && (tokens <= kUnsplit || seqs > kMostCounted))) return {0, false, seqs};
  const int64_t wide = seqs * hrows >= kManyRows ? kWideManyRows : kWide;
  if (!enough && tokens * head_dim <= wide) return {0, true, seqs};
  int64_t shares = (target + hrows - 1) / hrows;
  if (shares < seqs) shares = seqs;
  const int64_t items = shares + seqs;
  return {(int)shares, false, items < seqs * most ? items : seqs * most};
}

}  // namespace

// For any format and window: a smaller target or fewer attended tokens give no
// more items.
size_t kv_attention_workspace_bytes(int64_t seqs, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t tokens) {
  const Plan p = plan_of(kMostTarget, seqs, heads, kv_heads, head_dim, tokens);
  if (p.shares == 0) return 0;
  return (size_t)(p.items * heads) * (size_t)(head_dim + 2) * sizeof(float) + (size_t)seqs * sizeof(int2);
}

void launch_kv_attention(AttnArgs a, void* ws, hipStream_t stream) {
  a.head_tiles = (int32_t)head_tiles_of(a.heads, a.kv_heads);
  int64_t tokens = a.table_width << a.page_shift;
  if (a.window > 0 && tokens > (int64_t)a.window + kChunk) tokens = (int64_t)a.window + kChunk;
  const Plan p = plan_of(target_of(a.format, a.head_dim), a.seqs, a.heads, a.kv_heads, a.head_dim, tokens);
  a.shares = p.shares;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = a.part_o + p.items * a.heads * a.head_dim;
  a.part_plan = reinterpret_cast<int2*>(a.part_ml + p.items * a.heads * 2);
  const dim3 grid(a.kv_heads * a.head_tiles, (unsigned)p.items);
  if (a.format == W4_KV_BF16) launch_waves<W4_KV_BF16>(a, p.wide, grid, stream);
  else if (a.format == W4_KV_E4M3) launch_waves<W4_KV_E4M3>(a, p.wide, grid, stream);
  else launch_waves<W4_KV_Q4>(a, p.wide, grid, stream);
  if (a.shares > 0) {
    const dim3 rows(a.heads, (unsigned)a.seqs);
    if (a.head_dim == 64) kv_join_kernel<2><<<rows, 256, 0, stream>>>(a);
    else if (a.head_dim == 128) kv_join_kernel<4><<<rows, 256, 0, stream>>>(a);
    else kv_join_kernel<8><<<rows, 256, 0, stream>>>(a);
  }
}

}  // namespace w4
