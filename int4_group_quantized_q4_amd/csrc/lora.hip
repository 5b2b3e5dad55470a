// Low-rank adapters of many requests beside a projection:
//   out[t] = bf16(y[t] + s_i (x[t] A_i^T) B_i^T),  i = ids[t].
//
// Bound by memory: y is read and out written once, and every adapter that occurs
// is read once for each tile of its rows.  So rows of one adapter are gathered
// into tiles: of up to 64 by a sort of the ids, of up to 16 where there are at most
// 128 rows, among which every workgroup finds its tile's by itself.  The two products
// run on the 16x16x32 matrix cores with the factors' rows as the left and the tokens as
// the right operand, so that a lane ends with neighbouring r, or neighbouring n, of one
// token.
//   shrink  h = x A^T, fp32; a workgroup's waves take pieces of K, and other
//           workgroups parts of it where there are few tiles; the second kernel
//           joins their sums.
//   expand  h enters as three bf16 terms that hold its 24 bits (their products
//           with B are exact in the fp32 accumulators; one term would round h to
//           8 bits).  The terms lie one after another along the product's inner
//           dimension: 3 rank / 32 steps.
//
// Figures, of both kernels in a graph (K 4096; rows, N, rank, adapters): 1 of 2816 by
// 4096, rank 16: 8.7 us, two launches and as many round trips to memory.  64, 14336,
// 16, 48 of their own: 13.8 us, 25 MB, 1.8 TB/s; all of one adapter 11.6 us.  4090,
// 14336, 64, 7: 78 us; in a trace the sort 6, shrink 17, expand 56 (235 MB of y and out
// at 4.2 TB/s).

#include "common.h"
#include "serving.h"

namespace w4 {

namespace {

constexpr int kLoraThreads = 256;
constexpr int kWaves = kLoraThreads / 64;   // of the second product
constexpr int kTile = 64;           // rows of one adapter in a tile
// Up to as many rows need no sort (64-row pieces of the ids, one a lane).  With 256 in place of 128 that many rows took
// 39 us for 29 (rank 64, one adapter; a workgroup a row looks for its tile), and 64 of 48 adapters 14.5 for 13.8; with
// 64, 128 rows of 48 adapters 14.8 for 13.1.
constexpr int kDirectRows = 128;
// Their tiles: 64 rows of one adapter run side by side (rank 64, N 4096: 11.7 us; 29.9 in one tile, 24.8 in one with
// the groups' operands in registers together, which costs 64 rows of 48 adapters 1 us).
constexpr int kDirectTile = 16;
// Parts of K at most, and workgroups that the parts are to make: 64 rows of one adapter as above 34.8 us with 4 parts,
// 29.8 with 16, 35.5 with 32; 4090 rows 90 us with 128 workgroups, 77 with 256, 86 with 512.
constexpr int kMaxSplits = 16;
constexpr int kSplitGroups = 256;
constexpr int kSortThreads = 1024;
constexpr int kMaxAdapters = 4096;  // bins of the sort (and one for rows without)

struct TileInfo {
  int32_t id, start, count, pad;   // rows order[start .. start + count) of adapter id (-1: none)
};

struct LoraWork {
  int32_t* order;      // [rows], plan mode
  TileInfo* tiles;     // plan mode; null: each workgroup finds its own
  int32_t* n_tiles;
  float* part;         // [splits][rows][rank]
  int32_t splits, k_steps;   // parts of K, and 32-steps in a part
};

// ------------------------------------------------------------------ the sort
// Rows by adapter and tiles of them, by one workgroup: counts in LDS, scanned into
// offsets, then each row's place from its bin's counter.  The order of rows within
// an adapter does not matter (a row's result does not depend on its place).  A
// wave whose rows are all of one adapter, as in prompts, takes its places at once.
__global__ void __launch_bounds__(kSortThreads) lora_sort_kernel(const int32_t* ids, int rows, int adapters,
                                                                 LoraWork w) {
  __shared__ int s_count[kMaxAdapters + 1], s_tiles[kMaxAdapters + 1];
  __shared__ int s_wave[2][kSortThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, bins = adapters + 1;
  for (int b = tid; b < bins; b += kSortThreads) s_count[b] = 0;
  __syncthreads();
  const auto bin_of = [&](int t) {
    const int id = ids[t];
    return id < 0 || id >= adapters ? adapters : id;
  };
  // places in s_count[bin] for every lane's row (bin < 0: none)
  const auto place = [&](int bin) {
    const int first = __builtin_amdgcn_readfirstlane(bin);
    if (__ballot(bin != first) == 0) {
      int base = 0;
      if (lane == 0 && first >= 0) base = atomicAdd(&s_count[first], 64);
      return __builtin_amdgcn_readfirstlane(base) + lane;
    }
    return bin >= 0 ? atomicAdd(&s_count[bin], 1) : 0;
  };
  for (int t0 = wv * 64; t0 < rows; t0 += kSortThreads) place(t0 + lane < rows ? bin_of(t0 + lane) : -1);
  __syncthreads();
  // exclusive sums of rows and tiles over the bins
  const int per = (bins + kSortThreads - 1) / kSortThreads;
  const int b0 = min(bins, tid * per), b1 = min(bins, b0 + per);
  int n = 0, m = 0;
  for (int b = b0; b < b1; ++b) {
    n += s_count[b];
    m += (s_count[b] + kTile - 1) / kTile;
  }
  int n_up = n, m_up = m;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int x = __shfl_up(n_up, o, 64), y = __shfl_up(m_up, o, 64);
    if (lane >= o) {
      n_up += x;
      m_up += y;
    }
  }
  if (lane == 63) {
    s_wave[0][wv] = n_up;
    s_wave[1][wv] = m_up;
  }
  __syncthreads();
  int start = n_up - n, tile = m_up - m, tiles = 0;
  for (int v = 0; v < kSortThreads / 64; ++v) {
    if (v < wv) {
      start += s_wave[0][v];
      tile += s_wave[1][v];
    }
    tiles += s_wave[1][v];
  }
  for (int b = b0; b < b1; ++b) {
    const int c = s_count[b];
    s_count[b] = start;
    s_tiles[b] = tile;
    start += c;
    tile += (c + kTile - 1) / kTile;
  }
  if (tid == 0) *w.n_tiles = tiles;
  __syncthreads();
  for (int j = tid; j < tiles; j += kSortThreads) {
    int lo = 0, hi = bins;   // the last bin whose first tile is at most j: bins without rows share their follower's
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_tiles[mid] <= j) lo = mid;
      else hi = mid;
    }
    const int end = lo + 1 < bins ? s_count[lo + 1] : rows, at = s_count[lo] + (j - s_tiles[lo]) * kTile;
    w.tiles[j] = {lo < adapters ? lo : -1, at, min(kTile, end - at), 0};
  }
  __syncthreads();
  for (int t0 = wv * 64; t0 < rows; t0 += kSortThreads) {
    const int t = t0 + lane, bin = t < rows ? bin_of(t) : -1;
    const int at = place(bin);
    if (bin >= 0) w.order[at] = t;
  }
}

// The workgroup's tile: rows (of the call) in s_rows, adapter id and count; false
// where there is none.  Rows behind the count repeat the first one.
__device__ __forceinline__ bool find_tile(const LoraArgs& l, const LoraWork& w, int32_t* s_rows, int& id, int& count) {
  const int lane = threadIdx.x & 63, j = blockIdx.y;
  if (w.tiles) {
    if (j >= *w.n_tiles) return false;
    const TileInfo t = w.tiles[j];
    id = t.id;
    count = t.count;
    if (threadIdx.x < kTile) s_rows[lane] = w.order[t.start + (lane < count ? lane : 0)];
    __syncthreads();
    return true;
  }
  // The j-th row leads a tile if the number of rows of its adapter before it is a
  // multiple of 16; the tile is it and the next ones.
  int mine[kDirectRows / 64];
#pragma unroll
  for (int q = 0; q < kDirectRows / 64; ++q) {
    const int t = 64 * q + lane;
    mine[q] = t < l.rows ? l.ids[t] : -2;
    if (t < l.rows && (mine[q] < 0 || mine[q] >= l.adapters)) mine[q] = -1;
  }
  id = l.ids[j];
  if (id < 0 || id >= l.adapters) id = -1;
  int before = 0, all = 0, at[kDirectRows / 64];
#pragma unroll
  for (int q = 0; q < kDirectRows / 64; ++q) {
    const uint64_t same = __ballot(mine[q] == id);
    at[q] = mine[q] == id ? all + __builtin_popcountll(same & ((1ull << lane) - 1)) : -1;
    before += j >= 64 * q + 64 ? __builtin_popcountll(same)
              : j > 64 * q     ? __builtin_popcountll(same & ((1ull << (j & 63)) - 1))
                               : 0;
    all += __builtin_popcountll(same);
  }
  if (before % kDirectTile != 0) return false;
  count = min(kDirectTile, all - before);
  if (threadIdx.x < 64) {
    if (lane >= count) s_rows[lane] = j;
#pragma unroll
    for (int q = 0; q < kDirectRows / 64; ++q)
      if (at[q] >= before && at[q] < before + kDirectTile) s_rows[at[q] - before] = 64 * q + lane;
  }
  __syncthreads();
  return true;
}

// ---------------------------------------------------------------- x A^T
// RT tiles of 16 r; blockIdx.x: part of K + splits * (piece of the rank).  Each of
// the waves takes a piece of the part of K, for G groups of 16 tokens at once, so
// that A is loaded once for them; the pieces are summed in the order of the waves.
// A row's sums do not depend on the rows beside it.
template <int WAVES, int G, int RT>
__global__ void __launch_bounds__(64 * WAVES) lora_shrink_kernel(LoraArgs l, LoraWork w) {
  constexpr int kBatch = G == 1 ? 4 : 2;   // steps of K whose loads a wave issues together
  __shared__ int32_t s_rows[kTile];
  __shared__ f32x4 s_sum[WAVES][RT][64];
  int id, count;
  if (!find_tile(l, w, s_rows, id, count) || id < 0) return;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, c = lane >> 4;
  const int split = blockIdx.x % w.splits, r0 = (blockIdx.x / w.splits) * 16 * RT;
  const int s0 = split * w.k_steps, s1 = min(l.K / 32, s0 + w.k_steps);
  const int steps = max(0, s1 - s0), each = (steps + WAVES - 1) / WAVES;
  const int b = s0 + min(steps, wv * each), e = s0 + min(steps, (wv + 1) * each);
  const uint16_t* as[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)   // rows of r past the rank: the last one again, not stored
    as[i] = l.a + ((int64_t)id * l.rank + min(l.rank - 1, r0 + 16 * i + m)) * l.K + 8 * c;
  for (int g0 = 0; 16 * g0 < count; g0 += G) {
    f32x4 acc[G][RT];
    const uint16_t* xs[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      xs[g] = l.x + s_rows[min(16 * (g0 + g) + m, kTile - 1)] * l.x_stride + 8 * c;
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[g][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (int s = b; s < e; s += kBatch) {   // past the end the last step again, not added
      bf16x8 xv[kBatch][G], av[kBatch][RT];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int at = 32 * min(s + j, e - 1);
#pragma unroll
        for (int i = 0; i < RT; ++i) av[j][i] = *reinterpret_cast<const bf16x8*>(as[i] + at);
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (16 * (g0 + g) < count) xv[j][g] = *reinterpret_cast<const bf16x8*>(xs[g] + at);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (s + j < e) {
#pragma unroll
          for (int g = 0; g < G; ++g)
            if (16 * (g0 + g) < count) {
#pragma unroll
              for (int i = 0; i < RT; ++i) acc[g][i] = mfma16x16x32(av[j][i], xv[j][g], acc[g][i]);
            }
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (16 * (g0 + g) >= count) break;
      if (g0 + g > 0) __syncthreads();   // the sums of the group before are read
#pragma unroll
      for (int i = 0; i < RT; ++i) s_sum[wv][i][lane] = acc[g][i];
      __syncthreads();
      // 4 r of one token each
      if (wv < RT && 16 * (g0 + g) + m < count) {
        f32x4 sum = s_sum[0][wv][lane];
        for (int v = 1; v < WAVES; ++v) sum += s_sum[v][wv][lane];
        const int r = r0 + 16 * wv + 4 * c;
        if (r < l.rank)
          *reinterpret_cast<f32x4*>(w.part + ((int64_t)split * l.rows + s_rows[16 * (g0 + g) + m]) * l.rank + r) = sum;
      }
    }
  }
}

// ---------------------------------------------------------------- h B^T
// One of the three bf16 terms whose sum is v: truncated, the remainder truncated, the rest.
__device__ __forceinline__ uint16_t term_of(float v, int term) {
  const float hi = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
  if (term == 0) return (uint16_t)(__float_as_uint(v) >> 16);
  const float rest = v - hi;   // exact
  if (!(rest == rest)) return 0;   // v is not finite: the first term has it
  const float mid = __uint_as_float(__float_as_uint(rest) & 0xFFFF0000u);
  return term == 1 ? (uint16_t)(__float_as_uint(rest) >> 16) : bf16_rne(rest - mid);
}

// Where the inner dimension's chunk of 8 (term, 8 ch ..) lies: step and lane
// group.  Ranks of whole steps keep the terms of a chunk in successive steps, so
// that B's chunk is loaded once for the three; below 32 the terms follow one
// another, and B's chunk of a lane group is the same in all steps.
__device__ __forceinline__ int2 place_of(int term, int ch, int chunks) {
  if (chunks % 4 == 0) return {3 * (ch / 4) + term, ch % 4};
  const int q = term * chunks + ch;
  return {q / 4, q % 4};
}

// Between the products' layout, where a lane holds columns 8c.. and 32 + 8c.. of its
// own token, and memory's, where it holds columns 32 (m % 2) + 8c.. of the tokens m
// and m ^ 1 (the even one first), so that each load and store is of 128 bytes a row:
// the lanes of a pair give each other one piece.
__device__ __forceinline__ void swap_halves(u32x4 v[2]) {
  const bool odd = threadIdx.x & 1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t v0 = v[0][j], v1 = v[1][j];
    const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(odd ? v0 : v1), 0xB1, 0xF, 0xF, false);
    v[0][j] = odd ? got : v0;
    v[1][j] = odd ? v1 : got;
  }
}

// A wave takes `blocks` times 64 columns; blockIdx.x: which.  G groups of 16 tokens
// at a time have their terms in LDS.  STEPS of the inner dimension and LOADS chunks
// of B a lane: 1 and 1 (rank 8), 2 and 1 (16), 3 and 1 (32), 6 and 2 (64), 12 and 4
// (128); STEPS 0: any rank, B's chunks loaded at every step.
template <int G, int STEPS, int LOADS>
__global__ void __launch_bounds__(kLoraThreads) lora_expand_kernel(LoraArgs l, LoraWork w, int blocks) {
  extern __shared__ u32x4 s_terms[];   // [group][step][lane]: the operand's chunk of 8
  __shared__ int32_t s_rows[kTile];
  int id, count;
  if (!find_tile(l, w, s_rows, id, count)) return;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, c = lane >> 4;
  const int groups = (count + 15) / 16, chunks = l.rank / 8;
  const int steps = STEPS > 0 ? STEPS : (3 * chunks + 3) / 4;
  const int n0 = (blockIdx.x * kWaves + wv) * blocks * 64;
  if (id < 0) {
    if (l.out == l.y) return;
    for (int n = n0 + 8 * c; n < min(l.N, n0 + 64 * blocks); n += 32)
      for (int g = 0; g < groups; ++g)
        if (16 * g + m < count) {
          const int64_t row = s_rows[16 * g + m];
          *reinterpret_cast<u32x4*>(l.out + row * l.out_stride + n) =
              *reinterpret_cast<const u32x4*>(l.y + row * l.y_stride + n);
        }
    return;
  }
  const float scale = l.scaling ? l.scaling[id] : 1.0f;
  const uint16_t* bs = l.b + (int64_t)id * l.N * l.rank;
  // One block's chunks of B, and y of a round's tokens: asked for before the terms
  // of the first round are made, and, where registers allow (G == 1), while the
  // block before is computed.
  struct Block {
    bf16x8 v[LOADS][4];
    u32x4 old[G][2];
  };
  const auto load = [&](Block& k, int g0, int nb) {
    // rows n of the four left operands: the lane ends with twice 8 neighbouring columns
    if constexpr (STEPS > 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t* b = bs + (int64_t)min(nb + 32 * (i / 2) + 8 * (m / 4) + 4 * (i % 2) + m % 4, l.N - 1) * l.rank;
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
          k.v[j][i] = *reinterpret_cast<const bf16x8*>(b + 8 * ((4 * j + c) % (STEPS >= 3 ? 4 * LOADS : STEPS)));
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int token = 16 * (g0 + g) + (m & ~1) + h, n = nb + 32 * (m & 1) + 8 * c;
        if (token < count && n < l.N)
          k.old[g][h] = *reinterpret_cast<const u32x4*>(l.y + s_rows[token] * l.y_stride + n);
      }
  };
  Block now, next;
  if (n0 < l.N) load(now, 0, n0);
  for (int g0 = 0; g0 < groups; g0 += G) {
    const int here = min(G, groups - g0);
    if (g0 > 0) __syncthreads();   // the terms of the groups before are read
    for (int i = threadIdx.x; i < here * 16 * chunks; i += kLoraThreads) {
      const int token = i / chunks, ch = i - token * chunks;
      f32x4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      if (16 * g0 + token < count) {
        const f32x4* from = reinterpret_cast<const f32x4*>(w.part + (int64_t)s_rows[16 * g0 + token] * l.rank + 8 * ch);
        const int64_t pitch = l.rows * l.rank / 4;
#pragma unroll 4
        for (int s = 0; s < w.splits; ++s) {
          v[0] += from[s * pitch];
          v[1] += from[s * pitch + 1];
        }
      }
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = term_of(v[j / 2][2 * (j & 1)] * scale, term) |
                 ((uint32_t)term_of(v[j / 2][2 * (j & 1) + 1] * scale, term) << 16);
        const int2 at = place_of(term, ch, chunks);
        s_terms[((token / 16) * steps + at.x) * 64 + 16 * at.y + (token & 15)] = o;
      }
    }
    // the last step's lane groups behind the terms
    const int rest = 4 * steps - 3 * chunks;
    for (int i = threadIdx.x; i < here * 16 * rest; i += kLoraThreads) {
      const int g = i / (16 * rest), k = i - g * 16 * rest;
      s_terms[(g * steps + steps - 1) * 64 + 16 * (4 - rest) + k] = u32x4{0u, 0u, 0u, 0u};
    }
    __syncthreads();
    for (int p = 0; p < blocks; ++p) {
      const int nb = n0 + 64 * p;
      if (nb >= l.N) break;
      const bool more = p + 1 < blocks && nb + 64 < l.N;
      if (G == 1 && more) load(next, g0, nb + 64);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (g >= here) continue;
        f32x4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (STEPS > 0) {
          // lane groups behind the terms: zeros, as a NaN of B would not vanish
          constexpr int kRest = STEPS == 1 ? 1 : STEPS == 2 ? 2 : 0;
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const bf16x8 h = __builtin_bit_cast(bf16x8, s_terms[(g * STEPS + s) * 64 + lane]);
            const bool none = kRest > 0 && s == STEPS - 1 && c >= 4 - kRest;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[i] = mfma16x16x32(none ? bf16x8{} : now.v[s * LOADS / STEPS][i], h, acc[i]);
          }
        } else {
          for (int s = 0; s < steps; ++s) {
            // the chunk that place_of put at (s, c), or none
            int ch = chunks % 4 == 0 ? 4 * (s / 3) + c : 4 * s + c;
            const bool none = chunks % 4 != 0 && ch >= 3 * chunks;
            ch = none ? 0 : ch % chunks;
            const bf16x8 h = __builtin_bit_cast(bf16x8, s_terms[(g * steps + s) * 64 + lane]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int n = min(nb + 32 * (i / 2) + 8 * (m / 4) + 4 * (i % 2) + m % 4, l.N - 1);
              const bf16x8 v = *reinterpret_cast<const bf16x8*>(bs + (int64_t)n * l.rank + 8 * ch);
              acc[i] = mfma16x16x32(none ? bf16x8{} : v, h, acc[i]);
            }
          }
        }
        u32x4 o[2];
        swap_halves(now.old[g]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t was = now.old[g][j / 4][j % 4];
          const float lo = bf16_to_f32(was & 0xFFFFu) + acc[j / 2][2 * (j & 1)];
          const float hi = __uint_as_float(was & 0xFFFF0000u) + acc[j / 2][2 * (j & 1) + 1];
          o[j / 4][j % 4] = bf16_rne(lo) | ((uint32_t)bf16_rne(hi) << 16);
        }
        swap_halves(o);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int token = 16 * (g0 + g) + (m & ~1) + h, n = nb + 32 * (m & 1) + 8 * c;
          if (token < count && n < l.N) {
            u32x4* to = reinterpret_cast<u32x4*>(l.out + s_rows[token] * l.out_stride + n);
            // past the caches where there are many rows (the second product of 4090 rows of 14336 columns: 56
            // against 66 us, the call 78 against 90); few are what the next call reads
            if constexpr (G > 1) __builtin_nontemporal_store(o[h], to);
            else *to = o[h];
          }
        }
      }
      if (G > 1 && more) load(now, g0, nb + 64);
      else if (more) now = next;
    }
    if (g0 + G < groups && n0 < l.N) load(now, g0 + G, n0);
  }
}

template <int WAVES, int G>
void launch_shrink(const LoraArgs& l, const LoraWork& w, int rt, dim3 grid, hipStream_t stream) {
  if (rt == 1) lora_shrink_kernel<WAVES, G, 1><<<grid, 64 * WAVES, 0, stream>>>(l, w);
  else if (rt == 2) lora_shrink_kernel<WAVES, G, 2><<<grid, 64 * WAVES, 0, stream>>>(l, w);
  else lora_shrink_kernel<WAVES, G, 4><<<grid, 64 * WAVES, 0, stream>>>(l, w);
}

template <int G>
void launch_expand(const LoraArgs& l, const LoraWork& w, int blocks, dim3 grid, hipStream_t stream) {
  const int steps = (3 * (l.rank / 8) + 3) / 4;
  const size_t lds = (size_t)G * steps * 64 * sizeof(u32x4);
  switch (l.rank) {
    case 8: lora_expand_kernel<G, 1, 1><<<grid, kLoraThreads, lds, stream>>>(l, w, blocks); break;
    case 16: lora_expand_kernel<G, 2, 1><<<grid, kLoraThreads, lds, stream>>>(l, w, blocks); break;
    case 32: lora_expand_kernel<G, 3, 1><<<grid, kLoraThreads, lds, stream>>>(l, w, blocks); break;
    case 64: lora_expand_kernel<G, 6, 2><<<grid, kLoraThreads, lds, stream>>>(l, w, blocks); break;
    case 128: lora_expand_kernel<G, 12, 4><<<grid, kLoraThreads, lds, stream>>>(l, w, blocks); break;
    default: lora_expand_kernel<G, 0, 1><<<grid, kLoraThreads, lds, stream>>>(l, w, blocks);
  }
}

// Tiles that the rows make at most.
int64_t most_tiles(int64_t rows, int64_t adapters) {
  const int64_t each = rows / (rows > kDirectRows ? kTile : kDirectTile) + adapters + 1;
  return rows < each ? rows : each;
}

// Parts of K: enough workgroups for the chip where there are few tiles.
int splits_of(int64_t rows, int64_t K, int64_t adapters) {
  const int64_t want = kSplitGroups / most_tiles(rows, adapters), steps = K / 32;
  int64_t s = want < 1 ? 1 : want > kMaxSplits ? kMaxSplits : want;
  if (s > (steps + 3) / 4) s = (steps + 3) / 4;   // a step for each of the four waves
  return (int)s;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

size_t lora_workspace_bytes(int64_t rows, int64_t K, int64_t, int64_t adapters, int32_t rank) {
  size_t n = up16((size_t)splits_of(rows, K, adapters) * rows * rank * sizeof(float));
  if (rows > kDirectRows) n += up16((size_t)rows * 4) + (size_t)most_tiles(rows, adapters) * sizeof(TileInfo) + 16;
  return n;
}

void launch_lora(const LoraArgs& l, void* ws, hipStream_t stream) {
  LoraWork w{};
  char* at = static_cast<char*>(ws);
  const int64_t tiles = most_tiles(l.rows, l.adapters);
  w.splits = splits_of(l.rows, l.K, l.adapters);
  w.k_steps = (l.K / 32 + w.splits - 1) / w.splits;
  w.part = reinterpret_cast<float*>(at);
  at += up16((size_t)w.splits * l.rows * l.rank * sizeof(float));
  if (l.rows > kDirectRows) {
    w.order = reinterpret_cast<int32_t*>(at);
    at += up16((size_t)l.rows * 4);
    w.tiles = reinterpret_cast<TileInfo*>(at);
    w.n_tiles = reinterpret_cast<int32_t*>(at + (size_t)tiles * sizeof(TileInfo));
    lora_sort_kernel<<<1, kSortThreads, 0, stream>>>(l.ids, (int)l.rows, l.adapters, w);
  }
  const int r_tiles = (l.rank + 15) / 16;
  const int rt = r_tiles <= 1 ? 1 : r_tiles <= 2 ? 2 : 4;
  const unsigned groups_of_rows = (unsigned)(l.rows > kDirectRows ? tiles : l.rows);
  const dim3 shrink((unsigned)(w.splits * ((r_tiles + rt - 1) / rt)), groups_of_rows);
  if (l.rows <= kDirectRows) launch_shrink<4, 1>(l, w, rt, shrink, stream);
  else launch_shrink<8, 4>(l, w, rt, shrink, stream);
  const int64_t all = (l.N + 63) / 64;
  // 64-column blocks a wave: its terms serve all of them, where workgroups abound (64 rows of 48 adapters, N 14336:
  // 20.6 us with one, 15.6 with four; 64 rows of one, N 4096: 29.8 and 47.8)
  int64_t blocks = tiles * all / 4096;
  blocks = blocks >= 2 ? 4 : blocks >= 1 ? 2 : 1;
  const dim3 expand((unsigned)((all + kWaves * blocks - 1) / (kWaves * blocks)), groups_of_rows);
  // At most 64 KB of terms: four groups up to rank 168.
  if (l.rows <= kDirectRows) launch_expand<1>(l, w, (int)blocks, expand, stream);
  else if (l.rank <= 168) launch_expand<4>(l, w, (int)blocks, expand, stream);
  else launch_expand<2>(l, w, (int)blocks, expand, stream);
}

}  // namespace w4
