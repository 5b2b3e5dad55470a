// One token a row, drawn from its logits with a given uniform number.
//
// The kept tokens are a first piece of the order (logit descending, id ascending),
// so no sort of a row is needed.  Two kernels read the logits once:
//   scan  a workgroup for 16384 logits: their largest one, the sum of their
//         weights beside it (where the row needs the whole sum), and the
//         candidates: all logits from a bound up that at least `rank` of them reach,
//         the rank-th largest of the maxima of 256 groups;
//   draw  a workgroup a row.  All of the row's logits from the largest of the chunks'
//         bounds up are among the candidates: where that piece of the order decides
//         the filters, it is sorted in LDS, cut, and the draw is made among what is
//         left, in the order of the ids.  A row without filters needs no candidates:
//         the chunk in which the sums pass the number is read again.
// Rows for which that piece is too short (a nucleus of many thousand tokens) go
// through the row again, in the draw kernel: a radix select over the logits' order
// keys finds the last kept one by counts (top-k) and sums of weights (top-p).
//
// Weights are 2^((z - m) log2 e / T) in 64 bits.  Where they are added by atomics
// (the histogram of the top-p select) they are whole multiples of 2^-43, so that
// the sums do not depend on the order; elsewhere sums have a fixed order.

#include "common.h"
#include "serving.h"
#include "w4a16.h"

namespace w4 {

namespace {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kBins = 2048;
constexpr double kFixed = 0x1p43;   // 2^20 weights of at most 1 stay below 2^64

// 2^t for t <= 0 (2^-1100, that is 0, for a NaN): the series of 2^r to the 11th power,
// |r| <= 1/2, whose rest is below 1e-14 of it.
struct Series {
  double c[12];
  constexpr Series() : c() {
    double v = 1.0;
    for (int k = 0; k < 12; ++k) {
      c[k] = v;
      v *= 0.693147180559945309417232121458 / (k + 1);
    }
  }
};
__device__ __forceinline__ double exp2_f64(double t) {
  constexpr Series kSeries;
  t = __builtin_fmax(t, -1100.0);
  const double n = __builtin_rint(t), r = t - n;
  double v = kSeries.c[11];
#pragma unroll
  for (int k = 10; k >= 0; --k) v = __builtin_fma(v, r, kSeries.c[k]);
  return __builtin_ldexp(v, (int)n);
}

// Order keys: as unsigned numbers they compare as the logits do; zeros of both
// signs are one value; a NaN is the largest key.
constexpr uint32_t kNanKey = 0xFFFFFFFFu;
constexpr uint32_t kNegInfKey = 0x007FFFFFu;   // (0 stands for no logit)
constexpr uint32_t kPosInfKey = 0xFF800000u;

__device__ __forceinline__ uint32_t order_key(float z) {
  if (__builtin_isnan(z)) return kNanKey;
  const uint32_t b = __float_as_uint(z == 0.f ? 0.f : z);
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k); }

// A row's weights: exp((z - m) / T), 1 / T as given.
struct Weight {
  double top, per;   // m; log2 e / T
  bool infinite;     // m is +infinity: those weigh 1, all others 0
  __device__ __forceinline__ double operator()(uint32_t key) const {
    if (infinite) return key == kPosInfKey ? 1.0 : 0.0;
    return exp2_f64(((double)key_value(key) - top) * per);
  }
};

// The settings of a row, those that are off replaced by what they do not change.
struct Settings {
  int k;             // vocab: off
  double p, few;     // 1: off; 0: off
  float temperature; // 0: the largest logit
  double u;
  __device__ __forceinline__ bool greedy() const { return temperature == 0.f; }
  __device__ __forceinline__ bool filters(int n) const { return k < n || p < 1.0 || few > 0.0; }
  __device__ __forceinline__ Weight weight(uint32_t top) const {
    return {(double)key_value(top), 0x1.71547652b82fep+0 / (double)temperature, top == kPosInfKey};
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

__device__ __forceinline__ double shfl_f64(double v, int lane) {
  return __builtin_bit_cast(double, __shfl(__builtin_bit_cast(long long, v), lane, 64));
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __builtin_bit_cast(double, __shfl_xor(__builtin_bit_cast(long long, v), o, 64));
  return v;
}

template <typename T>
struct Row {
  const T* z;
  int n;
  __device__ __forceinline__ uint32_t key(int i) const {
    if constexpr (sizeof(T) == 2) return order_key(bf16_to_f32(z[i]));
    else return order_key(z[i]);
  }
};

struct Shared {
  unsigned long long bins[kBins];
  double seg[kSampleWaves];
  unsigned long long scan[kSampleWaves];
  uint32_t u32[kSampleWaves];
  int pick;
  unsigned long long above;
  int found;
};

// Sums of f over [lo, hi) in pieces of `piece` ids, one a wave, into s.seg; the
// piece in which the running sum first exceeds target, else the last one that is
// not 0; `before`: the sum of the pieces before it.
template <typename F>
__device__ int pick_piece(Shared& s, const F& f, int lo, int hi, int piece, double target, double& before,
                          double& total) {
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int b = min(hi, lo + wv * piece), e = min(hi, b + piece);
  double sum = 0;
  for (int i = b + lane; i < e; i += 64) sum += f(i);
  sum = wave_sum_f64(sum);
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
__device__ int find_id(Shared& s, const F& f, int lo, int hi, double share, double target, double& total) {
  int piece = piece_of(hi - lo);
  double before, ignored;
  if (share >= 0) {
    pick_piece(s, f, lo, hi, piece, 0.0, before, total);
    target = share * total;
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
      double c = v;
#pragma unroll
      for (int o = 1; o < 64; o *= 2) {
        const double x = shfl_f64(c, (lane - o) & 63);
        if (lane >= o) c += x;
      }
      const uint64_t past = __ballot(v > 0 && run + c > target), some = __ballot(v > 0);
      if (past) found = i0 + __builtin_ctzll(past);
      if (some) last = i0 + 63 - __builtin_clzll(some);
      run += shfl_f64(c, 63);
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
__device__ uint32_t radix_select(Shared& s, const R& row, const F& amount, unsigned long long need,
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

// A row by itself, whatever its filters.
template <typename T>
__device__ void whole_row(Shared& s, const SampleArgs& a, const Row<T>& row, int64_t r, const Settings& set,
                          const Weight& weight) {
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
    const auto amount = [&](uint32_t key, int i) {
      return kept(key, i) ? (unsigned long long)(weight(key) * kFixed + 0.5) : 0ull;
    };
    unsigned long long sum = 0;
    for (int i = tid; i < row.n; i += kSampleThreads) sum += amount(row.key(i), i);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
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
    const unsigned long long each = (unsigned long long)(weight(tp) * kFixed + 0.5);
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

// ---------------------------------------------------------------------- scan
constexpr int kPer = 16;                               // logits a thread
constexpr int kChunk = kSampleThreads * kPer;
constexpr int kGroups = 256;                           // of 4 threads each
constexpr int kListMost = 512;                         // candidates of a chunk
constexpr int kSortMost = 2048;                        // candidates of a row
constexpr int kSmallVocab = kSortMost;                 // up to here every logit is a candidate

struct ChunkInfo {
  double sum;        // of the weights beside top
  uint32_t top;      // largest key; 0: no logit above -infinity
  int32_t arg;       // the lowest id that has it
  uint32_t bound;    // every logit from this key up is in the list; 1: every one
  int32_t n;         // candidates; more than the list holds: it is not whole
};

int chunks_of(int64_t vocab) { return (int)((vocab + 7 + kChunk - 1) / kChunk); }   // a row starts inside 16 bytes
__host__ __device__ constexpr int list_most(int64_t vocab) { return vocab <= kSmallVocab ? kSmallVocab : kListMost; }

struct SampleWork {
  ChunkInfo* info;   // [rows][chunks]
  uint64_t* list;    // [rows][chunks][list_most]: key << 32 | ~id
  int chunks;
};

// The thread's logits of a chunk as keys (0: none), and their ids.  Chunks are cut at
// multiples of 16 bytes.
template <typename T>
struct Piece {
  static constexpr int kVec = 16 / sizeof(T);
  uint32_t key[kPer];
  int first;   // id of the chunk's first place
  __device__ __forceinline__ int id(int i) const {
    return first + (i / kVec * kSampleThreads + (int)threadIdx.x) * kVec + i % kVec;
  }
  __device__ __forceinline__ Piece(const T* z, int n, int chunk) {
    first = chunk * kChunk - (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
    u32x4 v[kPer / kVec];
#pragma unroll
    for (int j = 0; j < kPer / kVec; ++j) {
      const int at = id(j * kVec);
      if (at >= 0 && at + kVec <= n) {
        v[j] = *reinterpret_cast<const u32x4*>(z + at);
      } else {   // the row's first and last pieces; -infinity counts as no logit
        uint32_t e[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const bool in = at + i >= 0 && at + i < n;
          if constexpr (sizeof(T) == 2) e[i] = in ? z[at + i] : 0xFF80u;
          else e[i] = in ? __float_as_uint(z[at + i]) : 0xFF800000u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = sizeof(T) == 2 ? e[(2 * i) % kVec] | (e[(2 * i + 1) % kVec] << 16) : e[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t word = v[i / kVec][i % kVec * sizeof(T) / 4];
      const uint32_t bits = sizeof(T) == 2 ? (i % 2 ? word & 0xFFFF0000u : word << 16) : word;
      const uint32_t k = order_key(__uint_as_float(bits));
      key[i] = k == kNegInfKey ? 0u : k;
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kSampleThreads) sample_scan_kernel(SampleArgs a, SampleWork w) {
  __shared__ uint32_t s_top[kSampleWaves];
  __shared__ int s_arg, s_n;
  __shared__ double s_sum[kSampleWaves];
  __shared__ __align__(16) uint32_t s_group[kGroups];
  __shared__ uint32_t s_bound;
  const int64_t r = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const Piece<T> z(static_cast<const T*>(a.logits) + r * a.stride, a.vocab, blockIdx.x);
  const Settings set = settings_of(a, r);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = max(top, z.key[i]);
  const uint32_t mine = top;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
    if (o == 2 && (lane & 3) == 0) s_group[tid / 4] = top;
  }
  if (lane == 0) s_top[wv] = top;
  if (tid == 0) {
    s_arg = INT32_MAX;
    s_n = 0;
    s_bound = 1;
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kSampleWaves; ++v) top = max(top, s_top[v]);
  if (mine == top) {
    int arg = INT32_MAX;
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i)
      if (z.key[i] == top) arg = z.id(i);
    atomicMin(&s_arg, arg);
  }
  const bool sums = !set.greedy() && set.k >= a.vocab && (set.p < 1.0 || set.few == 0.0) && top != kNanKey;
  const bool lists = !set.greedy() && set.filters(a.vocab);
  // the bound: the rank-th largest of the groups' maxima (a lower one is a candidate
  // of the row only where `rank` of this chunk are above it)
  if (lists && a.vocab > kSmallVocab && tid < kGroups) {
    const int rank = set.k < a.vocab ? min(max(set.k, 16), kGroups) : 128;
    const uint32_t g = s_group[tid];
    int before = 0, some = 0;   // groups above this one; groups with a logit
#pragma unroll 4
    for (int j = 0; j < kGroups / 4; ++j) {
      const u32x4 o = reinterpret_cast<const u32x4*>(s_group)[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        before += o[i] > g || (o[i] == g && 4 * j + i < tid);
        some += o[i] > 0;
      }
    }
    if (before == min(rank, some) - 1) s_bound = g;
  }
  double sum = 0.0;
  if (sums && top > 0) {
    const Weight weight = set.weight(top);
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += weight(z.key[i]);
    sum = wave_sum_f64(sum);
  }
  if (lane == 0) s_sum[wv] = sum;
  __syncthreads();
  const uint32_t bound = a.vocab > kSmallVocab ? s_bound : 1u;
  const int64_t at = r * w.chunks + blockIdx.x;
  if (lists && mine >= bound) {
    uint64_t* list = w.list + at * list_most(a.vocab);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (z.key[i] >= bound) {
        const int n = atomicAdd(&s_n, 1);
        if (n < list_most(a.vocab)) list[n] = ((uint64_t)z.key[i] << 32) | (uint32_t)~z.id(i);
      }
  }
  __syncthreads();
  if (tid == 0) {
    sum = 0.0;
    for (int v = 0; v < kSampleWaves; ++v) sum += s_sum[v];
    w.info[at] = {sum, top, s_arg, bound, s_n};
  }
}

// ---------------------------------------------------------------------- draw
// v sorted in descending order, N (a power of two, 64 to 2048) of them in s_v, by
// the first N / 2 threads or fewer: bitonic, two values a thread; exchanges
// within a wave's 128 values need no barrier.
__device__ __forceinline__ void sort_descending(uint64_t* s_v, int N) {
  const int i = threadIdx.x;
  for (int size = 2; size <= N; size *= 2)
    for (int step = size / 2; step > 0; step /= 2) {
      if (step >= 64 || size == 2) __syncthreads();
      else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      if (i < N / 2) {
        const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
        const uint64_t x = s_v[lo], y = s_v[hi];
        const bool down = (lo & size) == 0;
        if ((x < y) == down) {
          s_v[lo] = y;
          s_v[hi] = x;
        }
      }
      if (step >= 64 && step / 2 < 64) __syncthreads();
    }
  __syncthreads();
}

// Inclusive running sums of the pairs (v0, v1) that each thread holds.
__device__ __forceinline__ void running_sums(double& v0, double& v1, double* s_wave, double& total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  double c = v0 + v1;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const double x = shfl_f64(c, (lane - o) & 63);
    if (lane >= o) c += x;
  }
  __syncthreads();
  if (lane == 63) s_wave[wv] = c;
  __syncthreads();
  double before = 0.0;
  total = 0.0;
  for (int v = 0; v < kSampleWaves; ++v) {
    if (v < wv) before += s_wave[v];
    total += s_wave[v];
  }
  const double upto = shfl_f64(c, (lane - 1) & 63);
  v0 += before + (lane > 0 ? upto : 0.0);
  v1 += v0;
}

union DrawShared {
  Shared whole;
  struct {
    uint64_t v[kSortMost];
    double sum[kSampleWaves];
    uint32_t top, bound;
    int n, kept, cut, token;
    bool ready;
  } draw;
};

template <typename T>
__global__ void __launch_bounds__(kSampleThreads) sample_draw_kernel(SampleArgs a, SampleWork w) {
  __shared__ DrawShared s;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const ChunkInfo* info = w.info + r * w.chunks;
  const Row<T> row{static_cast<const T*>(a.logits) + r * a.stride, a.vocab};
  const Settings set = settings_of(a, r);
  // the chunks' figures, up to 64 chunks a lane each
  uint32_t top = 0, bound = 0;
  int arg = INT32_MAX;
  bool whole = true;
  for (int c = lane; c < w.chunks; c += 64) {
    const ChunkInfo f = info[c];
    if (f.top > top) {
      top = f.top;
      arg = f.arg;
    }
    bound = max(bound, f.bound);
    whole = whole && f.n <= list_most(a.vocab);
  }
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const uint32_t t = (uint32_t)__shfl_xor((int)top, o, 64);
    const int g = __shfl_xor(arg, o, 64);
    if (t > top || (t == top && g < arg)) {
      top = t;
      arg = g;
    }
    bound = max(bound, (uint32_t)__shfl_xor((int)bound, o, 64));
  }
  whole = __ballot(!whole) == 0;
  if (top == kNanKey || top == 0 || set.greedy()) {
    if (tid == 0) {
      const bool none = top == kNanKey || top == 0;
      a.tokens[r] = none ? -1 : arg;
      if (a.logprobs) a.logprobs[r] = none ? __uint_as_float(0x7FC00000u) : 0.f;
    }
    return;
  }
  const Weight weight = set.weight(top);
  const bool sums = set.k >= a.vocab && (set.p < 1.0 || set.few == 0.0);
  double all = 0.0;   // of the whole row
  const auto chunk_sum = [&](int c) {
    const ChunkInfo f = info[c];
    return f.top == 0 ? 0.0 : f.sum * weight(f.top);
  };
  if (sums)
    for (int c = 0; c < w.chunks; ++c) all += chunk_sum(c);
  if (!set.filters(a.vocab)) {
    const double target = set.u * all;
    double run = 0.0, before = 0.0;
    int pick = -1, last = 0;
    double last_before = 0.0;
    for (int c = 0; c < w.chunks && pick < 0; ++c) {
      const double v = chunk_sum(c);
      if (run + v > target) {
        pick = c;
        before = run;
      }
      if (v > 0.0) {
        last = c;
        last_before = run;
      }
      run += v;
    }
    if (pick < 0) {
      pick = last;
      before = last_before;
    }
    const int first = pick * kChunk - (int)((reinterpret_cast<uintptr_t>(row.z) & 15u) / sizeof(T));
    double ignored;
    const int token = find_id(s.whole, [&](int i) { return weight(row.key(i)); }, max(first, 0),
                              min(a.vocab, first + kChunk), -1.0, target - before, ignored);
    if (tid == 0) {
      a.tokens[r] = token;
      if (a.logprobs) a.logprobs[r] = (float)log(weight(row.key(token)) / all);
    }
    return;
  }

  // candidates from the bound up
  if (tid == 0) s.draw.n = 0;
  __syncthreads();
  if (whole) {
    for (int c = tid / 64; c < w.chunks; c += kSampleWaves) {
      const int n = info[c].n;
      const uint64_t* list = w.list + (r * w.chunks + c) * list_most(a.vocab);
      for (int i = lane; i < n; i += 64) {
        const uint64_t v = list[i];
        if ((uint32_t)(v >> 32) >= bound) {
          const int at = atomicAdd(&s.draw.n, 1);
          if (at < kSortMost) s.draw.v[at] = v;
        }
      }
    }
  }
  __syncthreads();
  const int n = s.draw.n;
  bool ready = whole && n <= kSortMost && (set.k >= a.vocab || n >= set.k || bound == 1);
  int N = 64;
  while (N < n) N *= 2;
  if (ready) {
    for (int i = n + tid; i < N; i += kSampleThreads) s.draw.v[i] = 0;
    sort_descending(s.draw.v, N);
    // how many of the first ones stay
    const int i0 = 2 * tid, most = min(n, set.k);
    double w0 = i0 < most ? weight((uint32_t)(s.draw.v[i0] >> 32)) : 0.0;
    double w1 = i0 + 1 < most ? weight((uint32_t)(s.draw.v[i0 + 1] >> 32)) : 0.0;
    double c0 = w0, c1 = w1, total;
    running_sums(c0, c1, s.draw.sum, total);
    if (tid == 0) s.draw.kept = most;
    __syncthreads();
    if (set.p < 1.0) {
      const double need = set.p * (set.k < a.vocab || bound == 1 ? total : all);
      // the first place whose running sum reaches it
      if (c0 >= need && i0 < most) atomicMin(&s.draw.kept, i0 + 1);
      else if (c1 >= need && i0 + 1 < most) atomicMin(&s.draw.kept, i0 + 2);
      ready = total >= need;
    }
    if (set.few > 0.0) {
      if (i0 < most && w0 < set.few) atomicMin(&s.draw.kept, i0);
      else if (i0 + 1 < most && w1 < set.few) atomicMin(&s.draw.kept, i0 + 1);
    }
    __syncthreads();
    const int kept = s.draw.kept;
    // nothing below the bound would stay either
    ready = bound == 1 || kept < n || (set.k < a.vocab && kept == set.k) || (set.p < 1.0 && ready);
    ready = ready && kept > 0;
    if (ready) {
      // the kept ones in the order of their ids
      int M = 64;
      while (M < kept) M *= 2;
      const uint64_t x0 = i0 < kept ? s.draw.v[i0] : 0, x1 = i0 + 1 < kept ? s.draw.v[i0 + 1] : 0;
      __syncthreads();
      if (i0 < M) {   // ~id above the key: descending order is ascending in the id
        s.draw.v[i0] = x0 << 32 | x0 >> 32;
        s.draw.v[i0 + 1] = x1 << 32 | x1 >> 32;
      }
      if (tid == 0) {
        s.draw.token = INT32_MAX;
        s.draw.cut = -1;
      }
      sort_descending(s.draw.v, M);
      w0 = i0 < kept ? weight((uint32_t)s.draw.v[i0]) : 0.0;
      w1 = i0 + 1 < kept ? weight((uint32_t)s.draw.v[i0 + 1]) : 0.0;
      c0 = w0;
      c1 = w1;
      running_sums(c0, c1, s.draw.sum, total);
      const double target = set.u * total;
      if (w0 > 0.0) {
        if (c0 > target) atomicMin(&s.draw.token, i0);
        atomicMax(&s.draw.cut, i0);
      }
      if (w1 > 0.0) {
        if (c1 > target) atomicMin(&s.draw.token, i0 + 1);
        atomicMax(&s.draw.cut, i0 + 1);
      }
      __syncthreads();
      if (tid == 0) {
        const uint64_t v = s.draw.v[min(s.draw.token, s.draw.cut)];
        a.tokens[r] = (int32_t)~(uint32_t)(v >> 32);
        if (a.logprobs) a.logprobs[r] = (float)log(weight((uint32_t)v) / total);
      }
      return;
    }
  }
  __syncthreads();
  whole_row(s.whole, a, row, r, set, weight);
}

}  // namespace

size_t sample_workspace_bytes(int64_t rows, int64_t vocab) {
  return (size_t)rows * chunks_of(vocab) * (sizeof(ChunkInfo) + list_most(vocab) * sizeof(uint64_t));
}

void launch_sample(const SampleArgs& a, void* ws, hipStream_t stream) {
  SampleWork w{};
  w.chunks = chunks_of(a.vocab);
  w.list = static_cast<uint64_t*>(ws);
  w.info = reinterpret_cast<ChunkInfo*>(w.list + a.rows * w.chunks * list_most(a.vocab));
  const dim3 scan((unsigned)w.chunks, (unsigned)a.rows), draw((unsigned)a.rows);
  if (a.dtype == W4_OUT_F32) {
    sample_scan_kernel<float><<<scan, kSampleThreads, 0, stream>>>(a, w);
    sample_draw_kernel<float><<<draw, kSampleThreads, 0, stream>>>(a, w);
  } else {
    sample_scan_kernel<uint16_t><<<scan, kSampleThreads, 0, stream>>>(a, w);
    sample_draw_kernel<uint16_t><<<draw, kSampleThreads, 0, stream>>>(a, w);
  }
}

}  // namespace w4
