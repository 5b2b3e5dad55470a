// One token a row, drawn from its logits with a given uniform number.
//
// The kept tokens are a first piece of the order (logit descending, id ascending),
// so no sort of a row is needed.  Two kernels, which read the logits once:
//   scan  a workgroup for up to 16384 logits (a row's chunks are alike in size): their largest one, the sum of their
//         weights beside it (where the row needs the whole sum), and the
//         candidates: all logits from a bound up that at least `rank` of them reach,
//         the rank-th largest of the maxima of 256 groups, cut to its leading bits;
//   draw  a workgroup a row.  All of the row's logits from the largest of the chunks'
//         bounds up are among the candidates: where that piece of the order decides
//         the filters, it is cut, and the draw is made among what is left, in the
//         order of the ids.  Cuts and draw look for a place at which a running sum
//         reaches a border; the candidates are summed by 2048 bins of the order, and
//         only those of the bin with the border are compared (sorted are they where
//         that bin has more than 256: ties).  A row without filters needs no
//         candidates, only the 1024 logits in which the sums pass the number.
// A third one (rest) reads the rows again where that piece may be too short (a nucleus
// of thousands of tokens): several workgroups make histograms of the row's chunks' weights
// (and counts) over bins of a sixteenth of an octave, and the last one finds in them
// the bin of the last kept logit, reads the row once more for that bin's logits and one
// chunk of it for the draw, and cuts among them as above.  Where the bin holds too many
// (more than 2048: ties, long nuclei of the largest vocabularies) or a row has no
// histograms (mostly by a top_k of up to 64), one workgroup's radix select over the
// logits' order keys takes their place, and reads the row about a dozen times.
//
// Rows of 131072 fp32 logits, 64 of them, in us for the kernels: without filters
// scan 11.5 (of which the 64-bit powers take half: greedy rows 5.3), draw 5.0; top_k 50
// and top_p 0.95 8.7 and 10.9; top_k 1000 and top_p 0.9 10.2 and 14.2 (28.3 with all
// candidates sorted); top_p 0.9 15.0 and 9.8; rest without rows 2 to 4, with one that needs
// it 54 (of which one CU's reading of the row takes 18), with 64 such rows 64.  (With the
// histograms made by every scan that took 19 to 36 for all rows with a long filter.)
// 256 rows without filters: 34.5 and 5.3, 3.9 TB/s, the powers' instructions beside the
// loads.  What the radix select takes is far from that: a row with fewer allowed tokens
// than a top_k of 50, which misses the candidates because its few groups with a logit
// make the bound high, 556 for the three kernels, 64 such rows 762; rows of 262144 with
// temperature 1.5 and top_p 0.95, whose last bin holds some 3000 logits, 733 for one in
// rest, 1004 for 64.
//
// The second kernel's time is that of fetching its code as much as of running it (a
// workgroup passes through it once).  With the third kernel's code called from it, it
// took 8 us more, for a stack that no row used.
//
// Weights are 2^((z - m) log2 e / T) in 64 bits.  Where they are added by atomics they
// are whole multiples of 2^-52 (the candidates) or 2^-49 (the histograms) of the largest
// one, or as fine as the tokens' number allows (the radix select: of n of them 2^-63 n,
// down to 2^-52), so that the sums do not depend on the order; elsewhere sums have a fixed
// order.

#include "common.h"
#include "serving.h"
#include "w4a16.h"
#include "wave.h"

namespace w4 {

namespace {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kPer = 16;                               // logits a thread
constexpr int kChunk = kSampleThreads * kPer;          // most logits of a chunk
constexpr int kMostChunks = (1 << 20) / kChunk;        // one a lane
constexpr int kGroups = 256;                           // of 4 threads each
constexpr int kGroup = 4 * kPer;
constexpr int kRankSure = 64, kRankMost = 224;         // (the last groups' maxima say little about the bound)
constexpr int kListMost = 768;                         // candidates of a chunk
constexpr int kSortMost = 2048;                        // logits that are sorted
constexpr int kBinMost = 256;                          // candidates of a bin that are compared with one another
constexpr int kRestMost = 1024;                        // the same in the third kernel, which does not sort
constexpr int kSmallVocab = kSortMost;                 // up to here every logit is a candidate
constexpr int kFine = 1024;                            // bins of a 16th of an octave; the last one takes the rest
// Workgroups of the third kernel, up to one a chunk: each writes its XCD's L2 back, so more of them cost as well (54
// rows that need it 101 us with 512, 61 with 256; one row of 52 47.5 and 52, with 128 81 when 256 took 71).
constexpr int kRestGroups = 256;
constexpr int kBins = 2048;                            // of the radix select
constexpr double kFixed = 0x1p49;   // the 2^14 weights of a chunk's histogram, of at most 1, sum to at most 2^63

// 2^t for t <= 0; 0 below 2^-1074 and for a NaN.  The nearest whole number is what t
// leaves in the low bits of a large sum; 2^r, |r| <= 1/2, is 1 + r q(r) with the q of
// degree 10 that meets (2^r - 1) / r in the 11 Chebyshev points of [-1/2, 1/2].  With its
// roundings that is off by less than 2^-52 of the value, for as many instructions as the
// power series to the 11th power, which leaves out 2^-46.7 of it.
constexpr double kLarge = 0x1.8p52;
__device__ __forceinline__ double exp2_f64(double t) {
  constexpr double kPower[12] = {
      1.0,
      0x1.62e42fefa39efp-1, 0x1.ebfbdff82c598p-3, 0x1.c6b08d704a0c2p-5, 0x1.3b2ab6fba1ddap-7,
      0x1.5d87fe78a5276p-10, 0x1.430913096fd9fp-13, 0x1.ffcbfc670dcd4p-17, 0x1.62bfd47773353p-20,
      0x1.b524fae627834p-24, 0x1.e6063f7217bc6p-28, 0x1.e9d3fe3952179p-32};
  t = __builtin_fmax(t, -2000.0);
  const double sum = t + kLarge, r = t - (sum - kLarge);
  double v = kPower[11];
#pragma unroll
  for (int k = 10; k >= 0; --k) v = __builtin_fma(v, r, kPower[k]);
  return __builtin_ldexp(v, (int)(uint32_t)__builtin_bit_cast(uint64_t, sum));
}

// Order keys: as unsigned numbers they compare as the logits do; zeros of both
// signs are one value; a NaN is the largest key.
constexpr uint32_t kNanKey = 0xFFFFFFFFu;
constexpr uint32_t kNegInfKey = 0x007FFFFFu;   // (0 stands for no logit)
constexpr uint32_t kLowestKey = 0x00800000u;   // of the type's lowest value
constexpr uint32_t kPosInfKey = 0xFF800000u;

__device__ __forceinline__ uint32_t order_key(float z) {
  if (__builtin_isnan(z)) return kNanKey;
  const uint32_t b = __float_as_uint(z == 0.f ? 0.f : z);
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k); }

// The rank of a chunk's bound.  Up to 64 it is top_k: then the chunk with the largest
// bound has that many from there up, wherever the row's first ones lie.  Beyond, the
// rank at which about 1.5 top_k logits of the row are candidates if its chunks are
// alike (groups with one of e logits from the bound up: 256 (1 - exp(-e / 256)), as far
// as the chunk has 256); a row
// without top_k gets 64.  Ranks next to the number of groups make lists overflow.
__device__ __forceinline__ int rank_of(int k, int n, int chunk, int groups) {
  int rank = kRankSure;
  if (k <= kRankSure) rank = max(k, 16);
  else if (k < n) {
    const float e = 1.5f * (float)chunk * (float)k / (float)n, all = (float)(chunk / kGroup);
    rank = (int)fminf(fmaxf(all * (1.0f - __expf(-e / all)), kRankSure), kRankMost);
  }
  return max(1, min(rank, 7 * groups / 8));
}

// The least shift of a number below n that leaves less than 2048.  (A count of the leading zeros of 0 is not defined:
// an n of 1.)
__host__ __device__ constexpr int shift_of(int n) {
  const int bits = 32 - __builtin_clz((n - 1) | 1);
  return bits > 11 ? bits - 11 : 0;
}
static_assert(kSortMost == 2048 && shift_of(1) == 0 && shift_of(2048) == 0 && shift_of(2049) == 1 &&
              shift_of(1 << 20) == 9);

// A row's weights: 2^((z - m) log2 e / T).  (Beside an infinite m all but its equals
// are infinitely far below it, and weigh 0.)
struct Weight {
  float m;
  double top, per;   // m; log2 e / T
  __device__ __forceinline__ double of(float z) const {
    return exp2_f64(z == m ? 0.0 : ((double)z - top) * per);
  }
  __device__ __forceinline__ double operator()(uint32_t key) const { return of(key_value(key)); }
  // Sixteenths of an octave, whole ones: exact in fp32 below 2^24, and growing with z.
  __device__ __forceinline__ float steps(float z) const { return __builtin_rintf(z * (float)(16.0 * per)); }
};
// A weight in multiples of 2^-49 (the last bits of a number between 2^3 and 2^4), or of
// 2^-52 times another power of two.
__device__ __forceinline__ unsigned long long fixed_of(double w, double base = 0x1p52 / kFixed) {
  return __builtin_bit_cast(unsigned long long, w + base) - __builtin_bit_cast(unsigned long long, base);
}

// The settings of a row, those that are off replaced by what they do not change.
struct Settings {
  int k;             // vocab: off
  double p, few;     // 1: off; 0: off
  float temperature; // 0: the largest logit
  double u;
  __device__ __forceinline__ bool greedy() const { return temperature == 0.f; }
  __device__ __forceinline__ bool filters(int n) const { return k < n || p < 1.0 || few > 0.0; }
  // what a running sum has to exceed; a number of 1 takes the last kept token, however little it weighs
  __device__ __forceinline__ double target(double total) const { return u < 1.0 ? u * total : INFINITY; }
  // rows that need the sum of all weights, candidates, a histogram
  __device__ __forceinline__ bool sums(int n) const { return !greedy() && k >= n && (p < 1.0 || few == 0.0); }
  __device__ __forceinline__ bool lists(int n) const { return !greedy() && filters(n); }
  __device__ __forceinline__ bool bins(int n) const { return lists(n) && n > kSmallVocab && k > kRankSure; }
  __device__ __forceinline__ Weight weight(uint32_t top) const {
    const float m = key_value(top);
    return {m, (double)m, 0x1.71547652b82fep+0 / (double)temperature};
  }
};

__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t r) {
  Settings s;
  const float t = a.temperature ? a.temperature[r] : 1.0f;
  s.temperature = t > 0.f ? t : 0.f;
  const int k = a.top_k ? a.top_k[r] : 0;
  s.k = k <= 0 || k > a.vocab ? a.vocab : k;
  const float p = a.top_p ? a.top_p[r] : 1.0f;
  s.p = p < 1.0f ? (p > 0.f ? (double)p : 0.0) : 1.0;
  const float few = a.min_p ? a.min_p[r] : 0.0f;
  s.few = few > 0.f ? (few < 1.0f ? (double)few : 1.0) : 0.0;
  const float u = a.uniforms[r];
  s.u = u > 0.f ? (u < 1.0f ? (double)u : 1.0) : 0.0;
  return s;
}

template <typename T>
struct Row {
  const T* z;
  int n;
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(T) == 2) return bf16_to_f32(z[i]);
    else return z[i];
  }
  __device__ __forceinline__ uint32_t key(int i) const { return order_key(value(i)); }
};

// The thread's logits of a chunk (-infinity where there is none), and their ids: a wave
// has 1024 neighbouring ones, its lanes vectors of 16 bytes (at any multiple of the
// type's size).  A vector that would pass the row's end is moved back to end there,
// and what belongs to the vectors before it counts as none.
typedef u32x4 LooseVector __attribute__((aligned(2)));
constexpr int kWavePart = 64 * kPer;

template <typename T>
struct Piece {
  static constexpr int kVec = 16 / sizeof(T);
  float z[kPer];
  int first, end;   // id of the lane's first place; the row's length
  __device__ __forceinline__ int place(int j) const { return first + j * 64 * kVec; }
  __device__ __forceinline__ int id(int i) const { return min(place(i / kVec), end - kVec) + i % kVec; }
  // part: 1024 logits of the row
  struct Raw {
    u32x4 v[kPer / kVec];
  };
  static __device__ __forceinline__ int lane_first(int part) {
    return part * kWavePart + (int)(threadIdx.x & 63) * kVec;
  }
  static __device__ __forceinline__ Raw load(const Row<T>& row, int part) {   // rows of a vector and more
    Raw raw;
#pragma unroll
    for (int j = 0; j < kPer / kVec; ++j) {
      const int at = min(lane_first(part) + j * 64 * kVec, row.n - kVec);
      raw.v[j] = *reinterpret_cast<const LooseVector*>(row.z + at);
    }
    return raw;
  }
  __device__ __forceinline__ Piece(const Row<T>& row, int part) : first(lane_first(part)), end(row.n) {
    if (__builtin_expect(end < kVec, 0)) {   // less than a vector: the first lane's first places
      for (int i = 0; i < kPer; ++i)
        z[i] = i < kVec && first == 0 && id(i) >= 0 ? row.value(id(i)) : -INFINITY;
      return;
    }
    take(load(row, part), part);
  }
  __device__ __forceinline__ Piece(const Row<T>& row, int part, const Raw& raw) : first(lane_first(part)), end(row.n) {
    take(raw, part);
  }
  __device__ __forceinline__ void take(const Raw& raw, int part) {
    const u32x4(&v)[kPer / kVec] = raw.v;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t word = v[i / kVec][i % kVec * sizeof(T) / 4];
      z[i] = __uint_as_float(sizeof(T) == 4 ? word : i % 2 ? word & 0xFFFF0000u : word << 16);
    }
    if (part * kWavePart + kWavePart > end) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) z[i] = id(i) < place(i / kVec) ? -INFINITY : z[i];
    }
  }
};

// The wave's part of a chunk; chunks are of as many parts as there are for each, so that
// none is short; a wave without a part has one behind the row's end.
__device__ __forceinline__ int part_of(int chunk, int waves) {
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  return wv < waves ? chunk * waves + wv : (1 << 20) / kWavePart;
}

// f of every chunk of a row of a vector and more: the next two ones' loads are under way.
template <typename T, typename F>
__device__ __forceinline__ void for_chunks(const Row<T>& row, int chunks, int waves, const F& f) {
  using P = Piece<T>;
  const auto part = [&](int c) { return part_of(min(c, chunks - 1), waves); };
  typename P::Raw even = P::load(row, part(0)), odd = P::load(row, part(1));
  for (int c = 0; c < chunks; c += 2) {
    f(P(row, part(c), even));
    even = P::load(row, part(c + 2));
    if (c + 1 < chunks) f(P(row, part(c + 1), odd));
    odd = P::load(row, part(c + 3));
  }
}

// The piece's logits for which f holds, as key << 32 | ~id, behind the *n entries of a
// list that takes `most`; one atomic a wave.
template <typename T, typename F>
__device__ __forceinline__ void append(const Piece<T>& p, const F& f, int* n, uint64_t* list, int most) {
  uint32_t those = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) those |= f(p.z[i]) ? 1u << i : 0u;
  const int own = __builtin_popcount(those), upto = (int)wave_scan((int64_t)own);
  int at = 0;
  if ((threadIdx.x & 63) == 63 && upto > 0) at = atomicAdd(n, upto);
  at = __builtin_amdgcn_readlane(at, 63) + upto - own;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (those >> i & 1) {
      if (at < most) list[at] = ((uint64_t)order_key(p.z[i]) << 32) | (uint32_t)~p.id(i);
      ++at;
    }
}

struct ChunkInfo {
  double sum;        // of the weights beside top
  uint32_t top;      // largest key; 0: no logit above -infinity
  int32_t arg;       // the lowest id that has it
  uint32_t bound;    // every logit from this key up is in the list
  int32_t n;         // candidates; more than the list holds: it is not whole
};

__host__ __device__ constexpr int list_most(int64_t vocab) { return vocab <= kSmallVocab ? kSmallVocab : kListMost; }

struct SampleWork {
  ChunkInfo* info;             // [rows][chunks]
  double* part;                // [rows][chunks][kSampleWaves]: the waves' sums, beside the chunk's top
  int32_t *todo, *done;        // [rows]: left to the third kernel; its workgroups that have made their histograms
  uint64_t* list;              // [rows][chunks][list_most]: key << 32 | ~id
  unsigned long long* mass;    // [rows][chunks][kFine]
  uint16_t* count;             // [rows][chunks][kFine]
  int chunks, waves;           // parts of 1024 logits in a chunk
};

// ---------------------------------------------------------------------- scan
template <typename T>
__global__ void __launch_bounds__(kSampleThreads, 8) sample_scan_kernel(SampleArgs a, SampleWork w) {
  __shared__ uint32_t s_top[kSampleWaves];
  __shared__ int s_arg, s_n;
  __shared__ double s_sum[kSampleWaves];
  __shared__ uint32_t s_group[kGroups];
  __shared__ uint32_t s_bound;
  const int64_t r = blockIdx.y, at = r * w.chunks + blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const Row<T> row{static_cast<const T*>(a.logits) + r * a.stride, a.vocab};
  const Piece<T> piece(row, part_of(blockIdx.x, w.waves));
  const Settings set = settings_of(a, r);
  float m = piece.z[0];   // (a NaN stays)
#pragma unroll
  for (int i = 1; i < kPer; ++i) m = __builtin_elementwise_maximum(m, piece.z[i]);
  const uint32_t own = order_key(m), mine = own == kNegInfKey ? 0u : own;
  uint32_t top = quad_max(mine);
  if ((lane & 3) == 0) s_group[tid / 4] = top;
  top = wave_max_of_quads(top);
  const bool sums = set.sums(a.vocab), lists = set.lists(a.vocab);
  if (tid == 0) {
    s_arg = INT32_MAX;
    s_n = 0;
    s_bound = kLowestKey;
  }
  if (lists) __syncthreads();
  // the bound: the leading 18 bits of the rank-th largest of the groups' maxima, which
  // one wave finds bit by bit
  if (lists && a.vocab > kSmallVocab && wv == 0) {
    uint32_t g[kGroups / 64];
    int some = 0;   // groups with a logit
#pragma unroll
    for (int i = 0; i < kGroups / 64; ++i) {
      g[i] = s_group[64 * i + lane];
      some += __builtin_popcountll(__ballot(g[i] > 0));
    }
    const int rank = rank_of(set.k, a.vocab, w.waves * kWavePart, some);
    uint32_t bound = 0;
    for (uint32_t bit = 1u << 31; bit >= 1u << 14; bit >>= 1) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kGroups / 64; ++i) n += __builtin_popcountll(__ballot(g[i] >= (bound | bit)));
      if (n >= rank) bound |= bit;
    }
    if (lane == 0) s_bound = max(bound, kLowestKey);
  }
  // beside the wave's own top, for which it need not wait (256 rows without filters 39 us, 44 beside the chunk's)
  double sum = 0.0;
  if (top >= kPosInfKey) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += piece.z[i] == INFINITY ? 1.0 : 0.0;
  } else if (sums && top > 0) {
    const Weight weight = set.weight(top);
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += exp2_f64(((double)piece.z[i] - weight.top) * weight.per);
  }
  sum = wave_sum(sum);
  if (lane == 0) {
    s_top[wv] = top;
    s_sum[wv] = sum;
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kSampleWaves; ++v) top = max(top, s_top[v]);
  if (mine == top) {
    const float z = key_value(top);
    int arg = INT32_MAX;
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i)
      if (piece.z[i] == z) arg = piece.id(i);
    atomicMin(&s_arg, arg);
  }
  __syncthreads();
  const uint32_t bound = s_bound;
  if (lists && __ballot(mine >= bound)) {
    const float z = key_value(bound);
    append(piece, [&](float v) { return v >= z; }, &s_n, w.list + at * list_most(a.vocab), list_most(a.vocab));
  }
  __syncthreads();
  if (wv == 0) {
    const uint32_t part_top = lane < kSampleWaves ? s_top[lane] : 0u;
    const double part = part_top > 0 ? s_sum[lane] * set.weight(top)(part_top) : 0.0;
    sum = wave_sum(part);
    if (sums && lane < kSampleWaves) w.part[at * kSampleWaves + lane] = part;
    if (lane == 0) w.info[at] = {sum, top, s_arg, bound, s_n};
  }
}

// ---------------------------------------------------------------------- draw
// The first of 64 values (one a lane) at which their running sum exceeds target, the
// last positive one if none does; before: the sum of those in front of it.
__device__ __forceinline__ int pick_lane(double v, double target, double& before) {
  const double c = wave_scan(v);
  const uint64_t past = __ballot(v > 0.0 && c > target), some = __ballot(v > 0.0);
  const int pick = past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : 0;
  before = pick > 0 ? lane_value(c, pick - 1) : 0.0;
  return pick;
}

// The same for the settings' share of the whole sum.
__device__ __forceinline__ int pick_share(double v, const Settings& set, double& before, double& total) {
  total = lane_value(wave_scan(v), 63);
  return pick_lane(v, set.target(total), before);
}

// The id of a wave's part at which the running sum of f(logit, id) exceeds target, in
// the order of the ids (vector by vector, lane by lane), the last one with f > 0 if none
// does; share: f there.
template <typename T, typename F>
__device__ __forceinline__ int pick_in_part(const Piece<T>& p, const F& f, double target, double& share) {
  constexpr int kVec = Piece<T>::kVec;
  double own[kPer], chosen = 0.0, run = 0.0, before = 0.0;
  int vector = 0;
  bool found = false;
#pragma unroll
  for (int j = 0; j < kPer / kVec; ++j) {
    double mine = 0.0;
#pragma unroll
    for (int i = j * kVec; i < (j + 1) * kVec; ++i) {
      own[i] = f(p.z[i], p.id(i));
      mine += own[i];
    }
    const double sum = wave_sum(mine);
    if (sum > 0.0 && !found) {
      vector = j;
      chosen = mine;
      before = run;
      found = run + sum > target;
    }
    run += sum;
  }
  double in_front;
  const int lane = pick_lane(chosen, target - before, in_front);
  target -= before + in_front;
  int id = 0;
  run = 0.0;
  share = 0.0;
  found = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i / kVec == vector) {
      run += own[i];
      if (own[i] > 0.0 && !found) {
        id = p.id(i);
        share = own[i];
        found = run > target;
      }
    }
  share = lane_value(share, lane);
  return __builtin_amdgcn_readlane(id, lane);
}

// v0 (places 0 .. 1023) and v1 (1024 .. 2047) of all threads in descending order; N, a
// power of two from 64 up, is the number of places in use.  Bitonic: exchanges within
// a wave by moves between lanes, others through LDS.
__device__ __forceinline__ uint32_t across_u32(uint32_t v, int step) {   // of lane ^ 16 (rows swapped) or ^ 32 (halves)
  if (step == 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16) ? p[0] : p[1];
  }
  const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return (threadIdx.x & 32) ? p[0] : p[1];
}
// The value of lane ^ step, or one's own, whichever is larger (smaller).
__device__ __forceinline__ uint64_t exchange(uint64_t v, int step, bool larger) {
  const uint64_t other = step == 1   ? dpp_u64<0xB1>(v)                   // quad_perm [1,0,3,2]
                         : step == 2 ? dpp_u64<0x4E>(v)                   // quad_perm [2,3,0,1]
                         : step == 4 ? dpp_u64<0x1B>(dpp_u64<0x141>(v))   // half rows and quads mirrored
                         : step == 8 ? dpp_u64<0x128>(v)                  // row_ror 8
                                     : ((uint64_t)across_u32((uint32_t)(v >> 32), step) << 32) |
                                           across_u32((uint32_t)v, step);
  return (v > other) == larger ? v : other;
}
__device__ __forceinline__ uint64_t wave_merge(uint64_t v, bool descending) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int step = 32; step > 0; step /= 2) v = exchange(v, step, ((lane & step) == 0) == descending);
  return v;
}
__device__ __forceinline__ uint64_t wave_sort(uint64_t v, bool descending) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int size = 2; size < 64; size *= 2)
#pragma unroll
    for (int step = size / 2; step > 0; step /= 2)
      v = exchange(v, step, ((lane & step) == 0) == ((lane & size) == 0));
  return wave_merge(v, descending);
}
__device__ __forceinline__ void sort_descending(uint64_t* s_v, uint64_t& v0, uint64_t& v1, int N) {
  const int tid = threadIdx.x;
  const bool two = N > kSampleThreads;
  if (tid < N) v0 = wave_sort(v0, N == 64 || (tid & 64) == 0);
  if (two) v1 = wave_sort(v1, (tid & 64) == 0);
  for (int size = 128; size <= N; size *= 2) {
    if (size > kSampleThreads) {   // step 1024: the thread's own two
      const uint64_t a = v0, b = v1;
      v0 = a > b ? a : b;
      v1 = a > b ? b : a;
    }
    for (int step = min(size, kSampleThreads) / 2; step >= 64; step /= 2) {
      __syncthreads();
      s_v[tid] = v0;
      if (two) s_v[tid + kSampleThreads] = v1;
      __syncthreads();
      const uint64_t o0 = s_v[tid ^ step];
      v0 = (v0 > o0) == (((tid & step) == 0) == ((tid & size) == 0)) ? v0 : o0;
      if (two) {
        const uint64_t o1 = s_v[(tid ^ step) + kSampleThreads];
        v1 = (v1 > o1) == (((tid & step) == 0) == (((tid + kSampleThreads) & size) == 0)) ? v1 : o1;
      }
    }
    if (tid < N) v0 = wave_merge(v0, (tid & size) == 0);
    if (two) v1 = wave_merge(v1, ((tid + kSampleThreads) & size) == 0);
  }
}

// Inclusive running sums over the places: all v0, then all v1 (where the N places in
// use reach them).
__device__ __forceinline__ void running_sums(double& v0, double& v1, int N, double* s_wave, double& total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  total = 0.0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half == 1 && N <= kSampleThreads) break;
    const double c = wave_scan(half == 0 ? v0 : v1);
    __syncthreads();
    if (lane == 63) s_wave[wv] = c;
    __syncthreads();
    double before = total;
    for (int v = 0; v < kSampleWaves; ++v) {
      if (v < wv) before += s_wave[v];
      total += s_wave[v];
    }
    (half == 0 ? v0 : v1) = c + before;
  }
}

__device__ __forceinline__ int power_of_two(int n) { return n <= 64 ? 64 : 1 << (32 - __builtin_clz(n - 1)); }

// ------------------------------------------------- many candidates, not sorted
// The candidates of a row by 2048 bins in the order asked for: the bins' sums tell
// the bin in which the running sum reaches a border, and the candidates of that bin
// are compared with one another.
template <int MOST>   // of a bin that are compared
struct ReachShared {
  uint64_t v[kSortMost];
  unsigned long long bins[kSortMost];
  uint64_t bin_v[MOST];
  unsigned long long bin_x[MOST];
  unsigned long long scan[kSampleWaves], above;
  uint64_t last;
  int bin, n;
};

// Two candidates a thread with order values v (descending; their bins b ascend) and
// amounts x: the v of the first one at which the running sum of x is need(total) or
// more; 0 if need is, or if a bin holds too many.  2 us, whether the candidates are 50 or
// 1500; 128 of them compared with one another without bins took 3.5.
template <int MOST, typename F>
__device__ __forceinline__ uint64_t reach(ReachShared<MOST>& s, const uint64_t (&v)[2], const int (&b)[2],
                                          const unsigned long long (&x)[2], unsigned long long& total,
                                          const F& need_of) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  __syncthreads();   // what was read of the call before
#pragma unroll
  for (int i = 0; i < 2; ++i) s.bins[tid + i * kSampleThreads] = 0;
  if (tid == 0) {
    s.n = 0;
    s.last = 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (x[i] > 0) atomicAdd(&s.bins[b[i]], x[i]);
  __syncthreads();
  const unsigned long long first = s.bins[2 * tid], second = s.bins[2 * tid + 1];
  unsigned long long upto = wave_scan(first + second);
  if (lane == 63) s.scan[wv] = upto;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kSampleWaves; ++i) {
    const unsigned long long sum = s.scan[i];
    if (i < wv) upto += sum;
    total += sum;
  }
  const unsigned long long need = need_of(total);
  if (need == 0) return 0;
  const unsigned long long before = upto - first - second;
  if (before < need && upto >= need) {
    const bool in_first = before + first >= need;
    s.bin = 2 * tid + (in_first ? 0 : 1);
    s.above = in_first ? before : before + first;
  }
  __syncthreads();
  const int bin = s.bin;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (x[i] > 0 && b[i] == bin) {
      const int at = atomicAdd(&s.n, 1);
      if (at < MOST) {
        s.bin_v[at] = v[i];
        s.bin_x[at] = x[i];
      }
    }
  __syncthreads();
  const int n = s.n;
  if (n > MOST) return 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (x[i] > 0 && b[i] == bin) {
      unsigned long long run = s.above;
#pragma unroll 4
      for (int j = 0; j < n; ++j) run += s.bin_v[j] >= v[i] ? s.bin_x[j] : 0;
      if (run >= need && run - x[i] < need) s.last = v[i];
    }
  __syncthreads();
  return s.last;
}

// A weight in multiples of 2^-52, none of a positive one: 2048 of at most 1 stay below 2^64.
__device__ __forceinline__ unsigned long long finer_of(double w) {
  const unsigned long long x = __builtin_bit_cast(unsigned long long, w + 1.0) -
                               __builtin_bit_cast(unsigned long long, 1.0);
  return w > 0.0 && x == 0 ? 1 : x;
}

// ------------------------------------------------------- a row by its histograms
// The weights of a chunk's logits (and their number) by bins, beside its largest one.
// The last bin takes all the lower ones and is not used.
template <typename T>
__device__ __forceinline__ void add_to_bins(const Piece<T>& piece, const Weight& weight, unsigned long long* s_mass,
                                            uint32_t* s_count, bool counts) {
  const float ref = weight.steps(weight.m);
#pragma unroll
  for (int i = 0; i < kPer; i += 4) {   // four powers together share their coefficients
    double e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = exp2_f64(((double)piece.z[i + j] - weight.top) * weight.per);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = (int)fminf(ref - weight.steps(piece.z[i + j]), (float)(kFine - 1));
      const unsigned long long fixed = fixed_of(e[j]);
      if (fixed > 0 && b < kFine - 1) atomicAdd(&s_mass[b], fixed);
      if (counts && b < kFine - 1) atomicAdd(&s_count[b], 1u);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}
// Whether bins hold the row's weights.
__device__ __forceinline__ bool has_bins(const Weight& weight) {
  return weight.m < INFINITY && weight.per > 0.0 && __builtin_fabsf(weight.steps(weight.m)) < 0x1p22f;
}

struct WholeShared {
  ReachShared<kRestMost> order;
  double scale[kMostChunks], sums[kMostChunks];
  unsigned long long in_chunk[kMostChunks];
  int shift[kMostChunks];
  double scan[kSampleWaves];
  unsigned long long fixed[kSampleWaves];
  int bin, n;
  double above;
};

// The first bin at which the running sum of the threads' values (a bin each) reaches
// need (kFine: none does), and the sum before it.
__device__ __forceinline__ int reach_bin(WholeShared& s, double v, double need, double& above) {
  double c = v, none = 0.0, total;
  running_sums(c, none, kSampleThreads, s.scan, total);
  if (threadIdx.x == 0) s.bin = kFine;
  __syncthreads();
  if (v > 0.0 && c >= need) atomicMin(&s.bin, (int)threadIdx.x);
  __syncthreads();
  const int bin = s.bin;
  if ((int)threadIdx.x == bin) s.above = c - v;
  __syncthreads();
  above = s.above;
  return bin;
}

// The least key of a logit above -infinity for which f holds; f holds for all from some
// key on, the largest finite one's among them.  64 keys at a time, one a lane.
template <typename F>
__device__ __forceinline__ uint32_t least_key(const F& f) {
  uint32_t lo = kLowestKey;
  for (int shift = 26; shift >= 0; shift = shift > 6 ? shift - 6 : shift > 0 ? 0 : -1) {
    const uint64_t key = lo + ((uint64_t)(threadIdx.x & 63) << shift);
    const uint64_t no = __ballot(key < kPosInfKey && !f(key_value((uint32_t)key)));
    if (no) lo += ((uint32_t)(63 - __builtin_clzll(no)) << shift) + (shift == 0 ? 1 : 0);
    else if (shift == 0) break;
  }
  return lo;
}

// False: the histograms do not say, or a bin holds too many.
template <typename T>
__device__ __forceinline__ bool whole_row(WholeShared& s, const SampleArgs& a, const SampleWork& w, const Row<T>& row,
                                       int64_t r, const Settings& set, const Weight& weight, double all) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const float ref = weight.steps(weight.m);
  const ChunkInfo* info = w.info + r * w.chunks;
  const unsigned long long* mass = w.mass + r * w.chunks * kFine;
  const uint16_t* count = w.count + r * w.chunks * kFine;
  const bool use_k = set.k < a.vocab, use_p = set.p < 1.0;
  if (tid < w.chunks) {
    const uint32_t top = info[tid].top;
    const float shift = ref - weight.steps(key_value(top));
    s.scale[tid] = top == 0 ? 0.0 : weight(top) * (1.0 / kFixed);
    s.shift[tid] = top == 0 || !(shift < kFine) ? kFine : (int)shift;
    s.in_chunk[tid] = 0;
  }
  __syncthreads();
  const auto bin_of = [&](float z) { return (int)fminf(ref - weight.steps(z), (float)(kFine - 1)); };
  // the row's histograms, a bin a thread (the last bin is not used)
  double row_mass = 0.0, row_count = 0.0;
  if (tid < kFine - 1)
#pragma unroll 4
    for (int c = 0; c < w.chunks; ++c) {
      const int b = tid - s.shift[c], at = c * kFine + max(b, 0);   // loads without branches: several under way
      row_mass += b < 0 ? 0.0 : (double)mass[at] * s.scale[c];
      if (use_k) row_count += b < 0 ? 0.0 : (double)count[at];
    }
  // the logits of a bin, two a thread, with their weights and places among 2048 of the bin
  uint64_t v[2] = {0, 0};
  double wt[2];
  int place[2], listed = -1;
  const auto list = [&](int bin) {
    if (bin == listed) return true;
    listed = bin;
    const float lo = key_value(least_key([&](float z) { return bin_of(z) <= bin; }));
    const float end = bin > 0 ? key_value(least_key([&](float z) { return bin_of(z) < bin; })) : INFINITY;
    __syncthreads();
    if (tid == 0) s.n = 0;
    __syncthreads();
    for_chunks(row, w.chunks, w.waves, [&](const Piece<T>& p) {
      append(p, [&](float z) { return z >= lo && z < end; }, &s.n, s.order.v, kSortMost);
    });
    __syncthreads();
    if (s.n > kSortMost) return false;
    const float first = fminf(end, weight.m), scale = (float)(kSortMost - 1) / (first - lo);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = tid + i * kSampleThreads;
      v[i] = at < s.n ? s.order.v[at] : 0;
      const uint32_t key = (uint32_t)(v[i] >> 32);
      wt[i] = v[i] > 0 ? weight(key) : 0.0;
      place[i] = (int)fminf((first - key_value(key)) * scale, (float)(kSortMost - 1));
    }
    return true;
  };
  unsigned long long last = 0, x[2], total;   // last: of the last one kept, key << 32 | ~id; smaller ones are not
  const auto kept = [&]() {                   // the listed weights, those behind `last` left out
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = v[i] > 0 && v[i] >= last ? finer_of(wt[i]) : 0;
  };
  int bin = kFine - 1;   // the last one's
  double above, sum = all;
  if (use_k) {
    bin = reach_bin(s, row_count, (double)set.k, above);
    if (bin >= kFine - 1 || !list(bin)) return false;
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = v[i] > 0;
    last = reach(s.order, v, place, x, total,
                 [&](unsigned long long) { return (unsigned long long)set.k - (unsigned long long)above; });
    if (last == 0) return false;
    if (use_p) {
      kept();
      unsigned long long here = wave_sum(x[0] + x[1]);
      __syncthreads();
      if (lane == 0) s.fixed[wv] = here;
      __syncthreads();
      here = 0;
      for (int i = 0; i < kSampleWaves; ++i) here += s.fixed[i];
      double before = tid < bin ? row_mass : 0.0, none = 0.0;
      running_sums(before, none, kSampleThreads, s.scan, sum);
      sum += (double)here * 0x1p-52;
    }
  }
  if (use_p) {
    const double need = set.p * sum;
    const int reached = reach_bin(s, row_mass, need, above);
    if (reached >= kFine - 1 || reached > bin || !list(reached)) return false;
    bin = reached;
    kept();
    // the first place that reaches it, else the last one
    const double rest = __builtin_ceil((need - above) * 0x1p52);
    last = reach(s.order, v, place, x, total, [&](unsigned long long here) {
      return rest < (double)here ? (unsigned long long)__builtin_fmax(rest, 1.0) : here;
    });
    if (last == 0) return false;
  }
  if (set.few > 0.0) {
    const uint32_t least = least_key([&](float z) { return z >= weight.m || weight.of(z) >= set.few; });
    const int at = bin_of(key_value(least));
    if (at <= bin) {
      if (at >= kFine - 1 || !list(at)) return false;
      bin = at;
    }
    const unsigned long long from = (unsigned long long)least << 32;
    last = from > last ? from : last;
  }
  if (bin >= kFine - 1) return false;
  // the kept weights of each chunk: whole bins, and the listed ones
  kept();
  const int per = w.waves * kWavePart;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (x[i] > 0) atomicAdd(&s.in_chunk[(int)~(uint32_t)v[i] / per], x[i]);
  __syncthreads();
  for (int c = wv; c < w.chunks; c += kSampleWaves) {
    unsigned long long whole = 0;
    const int most = bin - s.shift[c];
#pragma unroll
    for (int i = 0; i < kFine / 64; ++i) {
      const unsigned long long m = mass[c * kFine + 64 * i + lane];
      whole += 64 * i + lane < most ? m : 0;
    }
    const double part = (double)wave_sum(whole) * s.scale[c] + (double)s.in_chunk[c] * 0x1p-52;
    if (lane == 0) s.sums[c] = part;
  }
  __syncthreads();
  double before, sum_kept;
  const int c = pick_share(lane < w.chunks ? s.sums[lane] : 0.0, set, before, sum_kept);
  const float last_z = key_value((uint32_t)(last >> 32));
  const int last_id = (int)~(uint32_t)last;   // (-1 where the key alone decides: as far as any id)
  const auto share = [&](float z, int id) {
    return z > last_z || (z == last_z && (uint32_t)id <= (uint32_t)last_id) ? weight.of(z) : 0.0;
  };
  const Piece<T> p(row, part_of(c, w.waves));
  double part = 0.0, in_front, weighs;
#pragma unroll
  for (int i = 0; i < kPer; ++i) part += share(p.z[i], p.id(i));
  part = wave_sum(part);
  if (lane == 0) s.scan[wv] = part;
  __syncthreads();
  const int picked = pick_lane(lane < kSampleWaves ? s.scan[lane] : 0.0, set.target(sum_kept) - before, in_front);
  if (wv != picked) return true;
  const int token = pick_in_part(p, share, set.target(sum_kept) - before - in_front, weighs);
  if (lane == 0) {
    a.tokens[r] = token;
    if (a.logprobs) a.logprobs[r] = (float)log(weighs / sum_kept);
  }
  return true;
}

// --------------------------------------------------- a row by a radix select
struct RadixShared {
  unsigned long long bins[kBins];
  double seg[kSampleWaves];
  unsigned long long scan[kSampleWaves];
  int pick;
  unsigned long long above;
  int found;
};

// Sums of f over [lo, hi) in pieces of `piece` ids, one a wave, into s.seg; the
// piece in which the running sum first exceeds target, else the last one that is
// not 0; `before`: the sum of the pieces before it.
template <typename F>
__device__ int pick_piece(RadixShared& s, const F& f, int lo, int hi, int piece, double target, double& before,
                          double& total) {
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int b = min(hi, lo + wv * piece), e = min(hi, b + piece);
  double sum = 0;
  for (int i = b + lane; i < e; i += 64) sum += f(i);
  sum = wave_sum(sum);
  __syncthreads();
  if (lane == 0) s.seg[wv] = sum;
  __syncthreads();
  double run = 0;
  int pick = -1;
  before = 0;
  int last = 0;
  double last_before = 0;
  for (int w = 0; w < kSampleWaves; ++w) {
    const double v = s.seg[w];
    if (pick < 0 && run + v > target) {
      pick = w;
      before = run;
    }
    if (v > 0) {
      last = w;
      last_before = run;
    }
    run += v;
  }
  total = run;
  if (pick < 0) {
    pick = last;
    before = last_before;
  }
  return pick;
}

__device__ __forceinline__ int piece_of(int n) { return ((n + kSampleWaves - 1) / kSampleWaves + 63) / 64 * 64; }

// The lowest id in [lo, hi) at which the running sum of f exceeds `share` of the
// whole sum (or `target`, where share is negative); the last one with f > 0 if
// none does.
template <typename F>
__device__ int find_id(RadixShared& s, const F& f, int lo, int hi, double share, double target, double& total) {
  int piece = piece_of(hi - lo);
  double before, ignored;
  if (share >= 0) {
    pick_piece(s, f, lo, hi, piece, 0.0, before, total);
    target = share < 1.0 ? share * total : INFINITY;
  }
  int w = pick_piece(s, f, lo, hi, piece, target, before, total);
  target -= before;
  lo = min(hi, lo + w * piece);
  hi = min(hi, lo + piece);
  piece = piece_of(hi - lo);
  w = pick_piece(s, f, lo, hi, piece, target, before, ignored);
  target -= before;
  lo = min(hi, lo + w * piece);
  hi = min(hi, lo + piece);
  // the last piece by one wave, 64 ids at a time
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    double run = 0;
    int found = -1, last = lo;
    for (int i0 = lo; i0 < hi && found < 0; i0 += 64) {
      const double v = i0 + lane < hi ? f(i0 + lane) : 0.0;
      const double c = wave_scan(v);
      const uint64_t past = __ballot(v > 0 && run + c > target), some = __ballot(v > 0);
      if (past) found = i0 + __builtin_ctzll(past);
      if (some) last = i0 + 63 - __builtin_clzll(some);
      run += lane_value(c, 63);
    }
    if (lane == 0) s.found = found >= 0 ? found : last;
  }
  __syncthreads();
  return s.found;
}

// The largest key t such that the amounts of the keys >= t sum to at least
// `need`; `above`: the sum over keys > t.  amount(key, i): 0 for ids that do not
// take part.  Digits of 11, 11 and 10 bits.
template <typename R, typename F>
__device__ uint32_t radix_select(RadixShared& s, const R& row, const F& amount, unsigned long long need,
                                 unsigned long long& above) {
  uint32_t prefix = 0;
  above = 0;
  for (int level = 0; level < 3; ++level) {
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
    const uint32_t held = level == 0 ? 0u : level == 1 ? 0xFFE00000u : 0xFFFFFC00u;
    const uint32_t mask = (1u << bits) - 1u;
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kSampleThreads) s.bins[b] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < row.n; i += kSampleThreads) {
      const uint32_t k = row.key(i);
      if ((k & held) == prefix) {
        const unsigned long long v = amount(k, i);
        if (v) atomicAdd(&s.bins[(k >> shift) & mask], v);
      }
    }
    __syncthreads();
    // two bins a thread, from the top down
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const unsigned long long hi = s.bins[kBins - 1 - 2 * tid], lo = s.bins[kBins - 2 - 2 * tid];
    unsigned long long c = hi + lo;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const unsigned long long x = __shfl_up(c, o, 64);
      if (lane >= o) c += x;
    }
    if (lane == 63) s.scan[wv] = c;
    if (tid == 0) s.pick = -1;
    __syncthreads();
    unsigned long long before = above + c - hi - lo;
    for (int w = 0; w < wv; ++w) before += s.scan[w];
    // exactly one thread's bins cross `need`
    if (before < need && before + hi + lo >= need) {
      const bool first = before + hi >= need;
      s.pick = kBins - 1 - 2 * tid - (first ? 0 : 1);
      s.above = first ? before : before + hi;
    }
    __syncthreads();
    if (s.pick < 0) return 0;   // less than `need` in all: every key
    prefix |= (uint32_t)s.pick << shift;
    above = s.above;
  }
  return prefix;
}

// For rows that have no histograms (a top_k of up to 64, infinities, extreme temperatures,
// numbers of 0 and 1) or whose histograms do not say (more than 2048 logits in the last bin).
template <typename T>
__device__ __forceinline__ void radix_row(RadixShared& s, const SampleArgs& a, const Row<T>& row, int64_t r,
                                          const Settings& set, const Weight& weight) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  // kept: keys above t, and ids up to `upto` at t
  uint32_t t = 0;
  int upto = row.n;
  double ignored;
  const auto kept = [&](uint32_t key, int i) { return key > t || (key == t && i <= upto); };
  if (set.k < row.n) {
    unsigned long long above;
    t = radix_select(s, row, [](uint32_t, int) { return 1ull; }, (unsigned long long)set.k, above);
    const double ties = (double)(set.k - (int64_t)above);
    upto = find_id(s, [&](int i) { return row.key(i) == t ? 1.0 : 0.0; }, 0, row.n, -1.0, ties - 1.0, ignored);
  }
  if (set.p < 1.0) {
    // as fine as the sum of those that may stay allows, which is at most 2^63: of up to 2048 multiples of 2^-52, of
    // 2^20 2^-43
    const double base = __builtin_ldexp(1.0, shift_of(min(set.k, row.n)));
    const auto amount = [&](uint32_t key, int i) {
      return kept(key, i) ? fixed_of(weight(key), base) : 0ull;
    };
    unsigned long long sum = 0;
    for (int i = tid; i < row.n; i += kSampleThreads) sum += amount(row.key(i), i);
    sum = wave_sum(sum);
    __syncthreads();
    if (lane == 0) s.scan[wv] = sum;
    __syncthreads();
    sum = 0;
    for (int w = 0; w < kSampleWaves; ++w) sum += s.scan[w];
    __syncthreads();
    const double part = set.p * (double)sum;
    const unsigned long long need = part > 1.0 ? (unsigned long long)__builtin_ceil(part) : 1ull;
    unsigned long long above;
    const uint32_t tp = radix_select(s, row, amount, need, above);
    const unsigned long long each = fixed_of(weight(tp), base);
    if (each > 0) {
      const double ties = (double)((need - above + each - 1) / each);
      upto = find_id(s, [&](int i) { return row.key(i) == tp ? 1.0 : 0.0; }, 0, row.n, -1.0, ties - 1.0, ignored);
      t = tp;
    }
  }
  const auto share = [&](int i) {
    const uint32_t key = row.key(i);
    if (!kept(key, i)) return 0.0;
    const double w = weight(key);
    return w < set.few ? 0.0 : w;
  };
  double total;
  const int token = find_id(s, share, 0, row.n, set.u, 0.0, total);
  if (tid == 0) {
    a.tokens[r] = token;
    if (a.logprobs) a.logprobs[r] = (float)log(weight(row.key(token)) / total);
  }
}

// ------------------------------------------------------------------ the draw
template <typename T>
__global__ void __launch_bounds__(kSampleThreads) sample_draw_kernel(SampleArgs a, SampleWork w) {
  __shared__ ReachShared<kBinMost> s;
  __shared__ double s_sum[kSampleWaves];
  __shared__ int s_n, s_kept, s_token, s_cut;
  uint64_t* const s_v = s.v;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const ChunkInfo* info = w.info + r * w.chunks;
  const Settings set = settings_of(a, r);
  // the chunks' figures, one a lane
  ChunkInfo mine{};
  if (lane < w.chunks) mine = info[lane];
  const uint32_t top = wave_max_of_quads(quad_max(mine.top));
  const uint32_t bound = wave_max_of_quads(quad_max(mine.bound));
  if (tid == 0) w.todo[r] = w.done[r] = 0;
  if (top == kNanKey || top == 0 || set.greedy()) {
    // the lowest id that has it: that of the first chunk
    const int arg = __builtin_amdgcn_readlane(mine.arg, __builtin_ctzll(__ballot(mine.top == top)));
    if (tid == 0) {
      const bool none = top == kNanKey || top == 0;
      a.tokens[r] = none ? -1 : arg;
      if (a.logprobs) a.logprobs[r] = none ? __uint_as_float(0x7FC00000u) : 0.f;
    }
    return;
  }
  const Weight weight = set.weight(top);
  double all = 0.0, before = 0.0;   // of the whole row's weights
  int chunk = 0;
  if (set.sums(a.vocab)) {
    chunk = pick_share(mine.top == 0 ? 0.0 : mine.sum * weight(mine.top), set, before, all);
  }
  if (!set.filters(a.vocab)) {
    if (tid >= 64) return;   // one wave reads on: the part of the chunk, and its logits
    const Row<T> row{static_cast<const T*>(a.logits) + r * a.stride, a.vocab};
    const double scale = weight(info[chunk].top);
    const double* parts = w.part + (r * w.chunks + chunk) * kSampleWaves;
    double in_front, share;
    const int part = pick_lane(lane < kSampleWaves ? parts[lane] * scale : 0.0, set.target(all) - before, in_front);
    const Piece<T> p(row, chunk * w.waves + part);
    const int token =
        pick_in_part(p, [&](float z, int) { return weight.of(z); }, set.target(all) - before - in_front, share);
    if (lane == 0) {
      a.tokens[r] = token;
      if (a.logprobs) a.logprobs[r] = (float)log(share / all);
    }
    return;
  }

  // candidates from the bound up
  const bool whole = __ballot(mine.n > list_most(a.vocab)) == 0;
  if (tid == 0) s_n = 0;
  __syncthreads();
  if (whole) {
    for (int c = tid / 64; c < w.chunks; c += kSampleWaves) {
      const int n = __builtin_amdgcn_readlane(mine.n, c);
      const uint64_t* list = w.list + (r * w.chunks + c) * list_most(a.vocab);
      for (int i = lane; i < n; i += 64) {
        const uint64_t v = list[i];
        if ((uint32_t)(v >> 32) >= bound) {
          const int at = atomicAdd(&s_n, 1);
          if (at < kSortMost) s_v[at] = v;
        }
      }
    }
  }
  __syncthreads();
  const int n = s_n;
  const bool complete = bound == kLowestKey;   // every logit is a candidate
  bool ready = whole && n <= kSortMost && (set.k >= a.vocab || n >= set.k || complete);
  if (ready) {
    const uint64_t v[2] = {tid < n ? s_v[tid] : 0, tid + kSampleThreads < n ? s_v[tid + kSampleThreads] : 0};
    // the bins of the values: from the largest one down to the bound, or (no bound) to weights of 2^-60
    const float range = complete ? (float)(60.0 / weight.per) : weight.m - key_value(bound);
    const float scale = (float)(kSortMost - 1) / range;
    unsigned long long x[2], total;
    double wt[2];
    int b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t key = (uint32_t)(v[i] >> 32);
      b[i] = (int)fminf((weight.m - key_value(key)) * scale, (float)(kSortMost - 1));
      wt[i] = v[i] > 0 ? weight(key) : 0.0;
      x[i] = v[i] > 0;
    }
    uint64_t last = 0;
    bool found = true, reached = false;   // no bin held too many; top_p falls among the candidates
    if (n > set.k) {
      last = reach(s, v, b, x, total, [&](unsigned long long) { return (unsigned long long)set.k; });
      found = last > 0;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = v[i] > 0 && v[i] >= last ? finer_of(wt[i]) : 0;
    if (found && set.p < 1.0) {
      last = reach(s, v, b, x, total, [&](unsigned long long sum) {
        const double need = set.p * (set.k < a.vocab || complete ? (double)sum : all * 0x1p52);
        reached = need <= (double)sum;
        return !reached ? 0ull : need > 1.0 ? min(sum, (unsigned long long)__builtin_ceil(need)) : 1ull;
      });
      found = !reached || last > 0;
    }
    if (found) {
      bool dropped = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (v[i] < last || wt[i] < set.few) {
          dropped |= v[i] > 0;
          x[i] = 0;
        }
      }
      // nothing below the bound would stay either
      ready = complete || set.k < a.vocab || reached || __syncthreads_or(dropped);
    }
    if (found && ready) {
      const int shift = shift_of(a.vocab);
      uint64_t by_id[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        by_id[i] = v[i] << 32 | v[i] >> 32;
        b[i] = (int)(~(uint32_t)v[i] >> shift) & (kSortMost - 1);
      }
      last = reach(s, by_id, b, x, total, [&](unsigned long long sum) {
        return set.u < 1.0 ? min(sum, (unsigned long long)(set.u * (double)sum) + 1) : sum;
      });
      found = last > 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (found && x[i] > 0 && by_id[i] == last) {
          a.tokens[r] = (int32_t)~(uint32_t)v[i];
          if (a.logprobs) a.logprobs[r] = (float)log(wt[i] / ((double)total * 0x1p-52));
        }
    }
    if (found && ready) return;
    ready = !found;   // sorted then
  }
  if (ready) {
    // First in the order of the logits: how many of the first ones stay; then those in
    // the order of their ids (~id above the key): the draw.
    const int i0 = tid, i1 = tid + kSampleThreads;
    uint64_t v0 = i0 < n ? s_v[i0] : 0, v1 = i1 < n ? s_v[i1] : 0;
    int most = min(n, set.k), N = power_of_two(n);
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      sort_descending(s_v, v0, v1, N);
      const int key_at = pass == 0 ? 32 : 0;
      const double w0 = i0 < most ? weight((uint32_t)(v0 >> key_at)) : 0.0;
      const double w1 = i1 < most ? weight((uint32_t)(v1 >> key_at)) : 0.0;
      double c0 = w0, c1 = w1, total;
      running_sums(c0, c1, N, s_sum, total);
      if (pass == 0) {
        if (tid == 0) {
          s_kept = most;
          s_token = INT32_MAX;
          s_cut = 0;
        }
        __syncthreads();
        if (set.p < 1.0) {
          const double need = set.p * (set.k < a.vocab || complete ? total : all);
          // the first place whose running sum reaches it
          if (i0 < most && c0 >= need) atomicMin(&s_kept, i0 + 1);
          if (i1 < most && c1 >= need) atomicMin(&s_kept, i1 + 1);
          ready = total >= need;
        }
        if (set.few > 0.0) {
          if (i0 < most && w0 < set.few) atomicMin(&s_kept, i0);
          if (i1 < most && w1 < set.few) atomicMin(&s_kept, i1);
        }
        __syncthreads();
        const int kept = s_kept;
        // nothing below the bound would stay either
        ready = complete || kept < n || (set.k < a.vocab && kept == set.k) || (set.p < 1.0 && ready);
        if (!ready) break;
        most = kept;
        N = power_of_two(kept);
        v0 = i0 < kept ? v0 << 32 | v0 >> 32 : 0;
        v1 = i1 < kept ? v1 << 32 | v1 >> 32 : 0;
      } else {
        const double target = set.target(total);
        if (w0 > 0.0) {
          if (c0 > target) atomicMin(&s_token, i0);
          atomicMax(&s_cut, i0);
        }
        if (w1 > 0.0) {
          if (c1 > target) atomicMin(&s_token, i1);
          atomicMax(&s_cut, i1);
        }
        __syncthreads();
        const int at = min(s_token, s_cut);
        if (at == i0 || at == i1) {
          a.tokens[r] = (int32_t)~(uint32_t)((at == i0 ? v0 : v1) >> 32);
          if (a.logprobs) a.logprobs[r] = (float)log((at == i0 ? w0 : w1) / total);
        }
        return;
      }
    }
  }
  if (tid == 0) w.todo[r] = 1;
}

// ---------------------------------------------------------------------- rest
struct BinsShared {
  unsigned long long mass[kFine];
  uint32_t count[kFine];
};
union RestShared {
  BinsShared bins;
  RadixShared radix;
  WholeShared whole;
};

template <typename T>
__global__ void __launch_bounds__(kSampleThreads) sample_rest_kernel(SampleArgs a, SampleWork w) {
  __shared__ RestShared s;
  __shared__ int s_last;
  const int64_t r = blockIdx.y;
  if (!w.todo[r]) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const ChunkInfo* info = w.info + r * w.chunks;
  const Row<T> row{static_cast<const T*>(a.logits) + r * a.stride, a.vocab};
  const Settings set = settings_of(a, r);
  ChunkInfo mine{};
  if (lane < w.chunks) mine = info[lane];
  const uint32_t top = wave_max_of_quads(quad_max(mine.top));
  const Weight weight = set.weight(top);
  const bool bins = set.bins(a.vocab) && has_bins(weight);
  if (bins) {
    // a histogram of every chunk, by the row's workgroups together; the last one goes on
    for (int c = blockIdx.x; c < w.chunks; c += gridDim.x) {
      const uint32_t chunk_top = info[c].top;
      if (chunk_top == 0) continue;
      __syncthreads();
      s.bins.mass[tid] = 0;
      s.bins.count[tid] = 0;
      __syncthreads();
      add_to_bins(Piece<T>(row, part_of(c, w.waves)), set.weight(chunk_top), s.bins.mass, s.bins.count,
                  set.k < a.vocab);
      __syncthreads();
      w.mass[(r * w.chunks + c) * kFine + tid] = s.bins.mass[tid];
      w.count[(r * w.chunks + c) * kFine + tid] = (uint16_t)s.bins.count[tid];
    }
    // Every wave's stores have reached the L2; one wave writes it back (all of them: 250 us more) and waits for that
    // before the count, and drops what its caches hold after it.
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (tid == 0) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
      __builtin_amdgcn_s_waitcnt(0);
      s_last = atomicAdd(&w.done[r], 1) == (int)gridDim.x - 1;
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      __builtin_amdgcn_s_waitcnt(0);
    }
    __syncthreads();
    if (!s_last) return;
  } else if (blockIdx.x > 0) {
    return;
  }
  double all = 0.0, before;
  if (set.sums(a.vocab)) {
    pick_share(mine.top == 0 ? 0.0 : mine.sum * weight(mine.top), set, before, all);
  }
  // (numbers of 0 and 1 ask for the first and the last weight, where multiples of 2^-49 will not do)
  if (bins && set.u > 0.0 && set.u < 1.0 && whole_row(s.whole, a, w, row, r, set, weight, all)) return;
  __syncthreads();
  radix_row(s.radix, a, row, r, set, weight);
}

size_t workspace_parts(int64_t rows, int64_t vocab, SampleWork& w, char* base) {
  const int parts = (int)((vocab + kWavePart - 1) / kWavePart);
  w.chunks = (parts + kSampleWaves - 1) / kSampleWaves;
  w.waves = (parts + w.chunks - 1) / w.chunks;
  const size_t n = (size_t)rows * w.chunks;
  w.list = reinterpret_cast<uint64_t*>(base);
  w.info = reinterpret_cast<ChunkInfo*>(w.list + n * list_most(vocab));
  w.part = reinterpret_cast<double*>(w.info + n);
  w.mass = reinterpret_cast<unsigned long long*>(w.part + n * kSampleWaves);
  const size_t bins = vocab > kSmallVocab ? n * kFine : 0;
  w.count = reinterpret_cast<uint16_t*>(w.mass + bins);
  w.todo = reinterpret_cast<int32_t*>(w.count + bins);
  w.done = w.todo + rows;
  return (size_t)(reinterpret_cast<char*>(w.done + rows) - base);
}

}  // namespace

size_t sample_workspace_bytes(int64_t rows, int64_t vocab) {
  SampleWork w{};
  return workspace_parts(rows, vocab, w, nullptr);
}

void launch_sample(const SampleArgs& a, void* ws, hipStream_t stream) {
  SampleWork w{};
  workspace_parts(a.rows, a.vocab, w, static_cast<char*>(ws));
  const dim3 scan((unsigned)w.chunks, (unsigned)a.rows), rows((unsigned)a.rows);
  const int64_t share = kRestGroups / a.rows, parts = share < 1 ? 1 : share < w.chunks ? share : w.chunks;
  const dim3 left((unsigned)parts, (unsigned)a.rows);
  // rows without filters, and rows whose logits are all candidates, are never left over
  const bool rest = (a.top_k || a.top_p || a.min_p) && a.vocab > kSmallVocab;
  const auto launch = [&](auto type) {
    using T = decltype(type);
    sample_scan_kernel<T><<<scan, kSampleThreads, 0, stream>>>(a, w);
    sample_draw_kernel<T><<<rows, kSampleThreads, 0, stream>>>(a, w);
    if (rest) sample_rest_kernel<T><<<left, kSampleThreads, 0, stream>>>(a, w);
  };
  if (a.dtype == W4_OUT_F32) launch(0.0f);
  else launch((uint16_t)0);
}

}  // namespace w4
