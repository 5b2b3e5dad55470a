// Low-rank adapters of many requests beside a projection:
//   out[t] = bf16(y[t] + s_i (x[t] A_i^T) B_i^T),  i = ids[t].
//
// Bound by memory: y is read and out written once, and every adapter that occurs
// is read once for each tile of its rows.  So rows of one adapter are gathered
// into tiles of up to 64 (by a sort of the ids; up to 64 rows every workgroup
// finds its tile's rows among them by itself), and the two products run on the
// 16x16x32 matrix cores with the factors' rows as the left and the tokens as the
// right operand, so that a lane ends with neighbouring r, or neighbouring n, of
// one token.
//   shrink  h = x A^T, fp32; the tile's groups of 16 tokens go to the four waves,
//           and what waves are left over, and other workgroups, take parts of K,
//           whose sums the second kernel joins.
//   expand  h enters as three bf16 terms that hold its 24 bits (their products
//           with B are exact in the fp32 accumulators; one term would round h to
//           8 bits).  The terms lie one after another along the product's inner
//           dimension: 3 rank / 32 steps, B's row read again at each.

#include "common.h"
#include "serving.h"

namespace w4 {

namespace {

constexpr int kLoraThreads = 256;
constexpr int kWaves = kLoraThreads / 64;
constexpr int kTile = 64;           // rows of one adapter in a tile
constexpr int kDirectRows = 64;     // up to as many rows need no sort
constexpr int kMaxSplits = 16;
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
  const int lane = threadIdx.x & 63, j = blockIdx.x;
  if (w.tiles) {
    if (j >= *w.n_tiles) return false;
    const TileInfo t = w.tiles[j];
    id = t.id;
    count = t.count;
    if (threadIdx.x < kTile) s_rows[lane] = w.order[t.start + (lane < count ? lane : 0)];
    __syncthreads();
    return true;
  }
  int mine = lane < l.rows ? l.ids[lane] : -2;
  if (lane < l.rows && (mine < 0 || mine >= l.adapters)) mine = -1;
  id = __builtin_amdgcn_readlane(mine, j);
  const uint64_t same = __ballot(mine == id);
  if (__builtin_ctzll(same) != j) return false;   // an earlier row's tile
  count = __builtin_popcountll(same);
  if (threadIdx.x < 64) {
    if (lane >= count) s_rows[lane] = j;
    if (mine == id) s_rows[__builtin_popcountll(same & ((1ull << lane) - 1))] = lane;
  }
  __syncthreads();
  return true;
}

// ---------------------------------------------------------------- x A^T
// RT tiles of 16 r; blockIdx.y: part of K + splits * (piece of the rank).
template <int RT>
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_kernel(LoraArgs l, LoraWork w) {
  __shared__ int32_t s_rows[kTile];
  __shared__ f32x4 s_sum[kWaves][RT][64];
  int id, count;
  if (!find_tile(l, w, s_rows, id, count) || id < 0) return;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, c = lane >> 4;
  const int split = blockIdx.y % w.splits, r0 = (blockIdx.y / w.splits) * 16 * RT;
  const int groups = (count + 15) / 16;
  const int per = groups == 1 ? 4 : groups == 2 ? 2 : 1;   // waves of a group of 16 tokens
  const int g = wv / per, part = wv % per;
  // The part of K is summed as (p0 + p1) + (p2 + p3) of its quarters, whichever
  // waves take them: a row's sums do not depend on the rows beside it.
  const int s0 = split * w.k_steps, s1 = min(l.K / 32, s0 + w.k_steps);
  const int steps = max(0, s1 - s0), each = (steps + 3) / 4;
  f32x4 sum[RT];
  if (g < groups) {
    const uint16_t* xs = l.x + s_rows[16 * g + m] * l.x_stride + 8 * c;
    const uint16_t* as[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)   // rows of r past the rank: the last one again, not stored
      as[i] = l.a + ((int64_t)id * l.rank + min(l.rank - 1, r0 + 16 * i + m)) * l.K + 8 * c;
    f32x4 half[RT];
    for (int q = part * (4 / per); q < (part + 1) * (4 / per); ++q) {
      f32x4 acc[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int b = s0 + min(steps, q * each), e = s0 + min(steps, (q + 1) * each);
      for (int s = b; s < e; ++s) {
        const bf16x8 xv = *reinterpret_cast<const bf16x8*>(xs + 32 * s);
#pragma unroll
        for (int i = 0; i < RT; ++i)
          acc[i] = mfma16x16x32(*reinterpret_cast<const bf16x8*>(as[i] + 32 * s), xv, acc[i]);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if (per == 4) sum[i] = acc[i];
        else if ((q & 1) == 0) half[i] = acc[i];
        else if (per == 2 || q == 1) sum[i] = half[i] + acc[i];
        else sum[i] += half[i] + acc[i];
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) s_sum[wv][i][lane] = sum[i];
  }
  __syncthreads();
  // 4 r of one token each, by the first wave of its group
  if (g < groups && part == 0 && 16 * g + m < count) {
    float* to = w.part + ((int64_t)split * l.rows + s_rows[16 * g + m]) * l.rank;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if (per == 4) sum[i] = (sum[i] + s_sum[wv + 1][i][lane]) + (s_sum[wv + 2][i][lane] + s_sum[wv + 3][i][lane]);
      else if (per == 2) sum[i] += s_sum[wv + 1][i][lane];
      const int r = r0 + 16 * i + 4 * c;
      if (r < l.rank) *reinterpret_cast<f32x4*>(to + r) = sum[i];
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

// A wave takes `pairs` times 32 columns; blockIdx.y: which.  G groups of 16
// tokens at a time have their terms in LDS.
template <int G>
__global__ void __launch_bounds__(kLoraThreads) lora_expand_kernel(LoraArgs l, LoraWork w, int pairs) {
  extern __shared__ u32x4 s_terms[];   // [group][step][lane]: the operand's chunk of 8
  __shared__ int32_t s_rows[kTile];
  int id, count;
  if (!find_tile(l, w, s_rows, id, count)) return;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, c = lane >> 4;
  const int groups = (count + 15) / 16, chunks = l.rank / 8, steps = (3 * chunks + 3) / 4;
  const int n0 = (blockIdx.y * kWaves + wv) * pairs * 32;
  if (id < 0) {
    if (l.out == l.y) return;
    for (int p = 0; p < pairs; ++p) {
      const int n = n0 + 32 * p + 8 * c;
      if (n >= l.N) break;
      for (int g = 0; g < groups; ++g)
        if (16 * g + m < count) {
          const int64_t row = s_rows[16 * g + m];
          *reinterpret_cast<u32x4*>(l.out + row * l.out_stride + n) =
              *reinterpret_cast<const u32x4*>(l.y + row * l.y_stride + n);
        }
    }
    return;
  }
  const float scale = l.scaling ? l.scaling[id] : 1.0f;
  const uint16_t* bs = l.b + (int64_t)id * l.N * l.rank;
  for (int g0 = 0; g0 < groups; g0 += G) {
    const int here = min(G, groups - g0);
    if (g0 > 0) __syncthreads();   // the terms of the groups before are read
    for (int i = threadIdx.x; i < here * steps * 64; i += kLoraThreads) {
      const int q = 4 * (i / 64 % steps) + (i & 63) / 16, token = 16 * (g0 + i / 64 / steps) + (i & 15);
      u32x4 o = {0u, 0u, 0u, 0u};
      if (q < 3 * chunks && token < count) {
        const int term = q / chunks;
        const float* from = w.part + (int64_t)s_rows[token] * l.rank + 8 * (q - term * chunks);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = from[j];
        for (int s = 1; s < w.splits; ++s) {
          from += l.rows * l.rank;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += from[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = term_of(v[2 * j] * scale, term) | ((uint32_t)term_of(v[2 * j + 1] * scale, term) << 16);
      }
      s_terms[i] = o;
    }
    __syncthreads();
    for (int p = 0; p < pairs; ++p) {
      const int nb = n0 + 32 * p;
      if (nb >= l.N) break;
      // rows n of the two left operands: the lane ends with 8 neighbouring columns
      const int row0 = nb + 8 * (m / 4) + m % 4;
      const uint16_t* b0 = bs + (int64_t)min(row0, l.N - 1) * l.rank;
      const uint16_t* b1 = bs + (int64_t)min(row0 + 4, l.N - 1) * l.rank;
      const int n = nb + 8 * c;
      u32x4 old[G];
      f32x4 acc[G][2];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        acc[g][0] = acc[g][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (n < l.N && 16 * (g0 + g) + m < count)
          old[g] = *reinterpret_cast<const u32x4*>(l.y + s_rows[16 * (g0 + g) + m] * l.y_stride + n);
      }
      for (int s = 0; s < steps; ++s) {
        const int q = 4 * s + c;
        const int at = q < 3 * chunks ? 8 * (q % chunks) : 0;   // (past the end: times the zeros of s_terms)
        bf16x8 v0 = *reinterpret_cast<const bf16x8*>(b0 + at), v1 = *reinterpret_cast<const bf16x8*>(b1 + at);
        if (q >= 3 * chunks) v0 = v1 = bf16x8{};   // a NaN there would not vanish
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (g < here) {
            const bf16x8 h = __builtin_bit_cast(bf16x8, s_terms[(g * steps + s) * 64 + lane]);
            acc[g][0] = mfma16x16x32(v0, h, acc[g][0]);
            acc[g][1] = mfma16x16x32(v1, h, acc[g][1]);
          }
      }
      if (n < l.N) {
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (16 * (g0 + g) + m < count) {
            u32x4 o;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x4 d = acc[g][j / 2];
              const float lo = bf16_to_f32(old[g][j] & 0xFFFFu) + d[2 * (j & 1)];
              const float hi = __uint_as_float(old[g][j] & 0xFFFF0000u) + d[2 * (j & 1) + 1];
              o[j] = bf16_rne(lo) | ((uint32_t)bf16_rne(hi) << 16);
            }
            *reinterpret_cast<u32x4*>(l.out + s_rows[16 * (g0 + g) + m] * l.out_stride + n) = o;
          }
      }
    }
  }
}

// Tiles that the rows make at most.
int64_t most_tiles(int64_t rows, int64_t adapters) {
  const int64_t each = rows / kTile + adapters + 1;
  return rows < each ? rows : each;
}

// Parts of K: enough workgroups for the chip where there are few tiles.
int splits_of(int64_t rows, int64_t K, int64_t adapters) {
  const int64_t want = 512 / most_tiles(rows, adapters), steps = K / 32;
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
  const dim3 shrink(groups_of_rows, (unsigned)(w.splits * ((r_tiles + rt - 1) / rt)));
  if (rt == 1) lora_shrink_kernel<1><<<shrink, kLoraThreads, 0, stream>>>(l, w);
  else if (rt == 2) lora_shrink_kernel<2><<<shrink, kLoraThreads, 0, stream>>>(l, w);
  else lora_shrink_kernel<4><<<shrink, kLoraThreads, 0, stream>>>(l, w);
  const int64_t all = (l.N + 31) / 32;
  int64_t pairs = tiles * all / 4096;
  pairs = pairs < 1 ? 1 : pairs > 8 ? 8 : pairs;
  const int steps = (3 * (l.rank / 8) + 3) / 4;
  const int64_t groups = ((l.rows < kTile ? l.rows : kTile) + 15) / 16;
  const dim3 expand(groups_of_rows, (unsigned)((all + kWaves * pairs - 1) / (kWaves * pairs)));
  // at most 64 KB of terms: four groups up to rank 168, else two
  const size_t group_bytes = (size_t)steps * 64 * 16;
  const size_t most = steps <= 16 ? 4 : 2, lds = (size_t)(groups < (int64_t)most ? (size_t)groups : most) * group_bytes;
  if (steps <= 16) lora_expand_kernel<4><<<expand, kLoraThreads, lds, stream>>>(l, w, (int)pairs);
  else lora_expand_kernel<2><<<expand, kLoraThreads, lds, stream>>>(l, w, (int)pairs);
}

}  // namespace w4
