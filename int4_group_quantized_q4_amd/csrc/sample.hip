// One token a row, drawn from its logits with a given uniform number.
//
// The kept tokens are a first piece of the order (logit descending, id
// ascending): all above a logit t and the first few ids at t.  So no sort is
// needed: a logit's order key is its 32 bits made monotonic, a radix select over
// the keys finds t by counts (top-k) and by sums of weights (top-p), and the draw
// is a search over the running sums in the order of the ids.
//
// Weights are exp in 64 bits.  Where they are added by atomics (the histogram of
// the top-p select) they are whole multiples of 2^-43, so that the sums do not
// depend on the order; elsewhere sums have a fixed order.

#include "common.h"
#include "serving.h"
#include "w4a16.h"

namespace w4 {

namespace {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kBins = 2048;
constexpr double kFixed = 0x1p43;   // 2^20 weights of at most 1 stay below 2^64

// Order keys: as unsigned numbers they compare as the logits do; zeros of both
// signs are one value; a NaN is the largest key.
constexpr uint32_t kNanKey = 0xFFFFFFFFu;
constexpr uint32_t kNegInfKey = 0x007FFFFFu;
constexpr uint32_t kPosInfKey = 0xFF800000u;

__device__ __forceinline__ uint32_t order_key(float z) {
  if (__builtin_isnan(z)) return kNanKey;
  const uint32_t b = __float_as_uint(z == 0.f ? 0.f : z);
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k); }

// A row's weights: exp((z - m) / T), 1 / T as given.
struct Weight {
  double top, inv_t;
  bool infinite;   // m is +infinity: those weigh 1, all others 0
  __device__ __forceinline__ double operator()(uint32_t key) const {
    if (infinite) return key == kPosInfKey ? 1.0 : 0.0;
    if (key == kNegInfKey) return 0.0;
    return exp(((double)key_value(key) - top) * inv_t);
  }
};

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

// The lowest id in [0, n) at which the running sum of f exceeds `share` of the
// whole sum (or `target`, where share is negative); the last one with f > 0 if
// none does.
template <typename F>
__device__ int find_id(Shared& s, const F& f, int n, double share, double target, double& total) {
  int lo = 0, hi = n, piece = piece_of(n);
  double before, ignored;
  if (share >= 0) {
    pick_piece(s, f, lo, hi, piece, 0.0, before, total);
    target = share * total;
  }
  // the sums in s.seg are of the same pieces: picked again with the target known
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

template <typename T>
__global__ void __launch_bounds__(kSampleThreads) sample_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const Row<T> row{static_cast<const T*>(a.logits) + r * a.stride, a.vocab};
  uint32_t top = 0;
  for (int i = tid; i < row.n; i += kSampleThreads) top = max(top, row.key(i));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
  if (lane == 0) s.u32[wv] = top;
  __syncthreads();
  for (int w = 0; w < kSampleWaves; ++w) top = max(top, s.u32[w]);

  if (top == kNanKey || top <= kNegInfKey) {
    if (tid == 0) {
      a.tokens[r] = -1;
      if (a.logprobs) a.logprobs[r] = __uint_as_float(0x7FC00000u);
    }
    return;
  }
  const float temperature = a.temperature ? a.temperature[r] : 1.0f;
  const bool greedy = !(temperature > 0.f);
  int k = a.top_k ? a.top_k[r] : 0;
  k = greedy ? 1 : k <= 0 || k > row.n ? row.n : k;
  const float p = a.top_p && !greedy ? a.top_p[r] : 1.0f;
  float few = a.min_p && !greedy ? a.min_p[r] : 0.0f;
  few = few > 1.0f ? 1.0f : few;
  const bool use_p = p < 1.0f, use_min = few > 0.0f;
  float u = a.uniforms[r];
  u = u > 0.f ? (u < 1.0f ? u : 1.0f) : 0.f;
  const Weight weight{(double)key_value(top), greedy ? 1.0 : 1.0 / (double)temperature, top == kPosInfKey};

  // kept: keys above t, and ids up to `upto` at t
  uint32_t t = 0;
  int upto = row.n;
  double ignored;
  const auto kept = [&](uint32_t key, int i) { return key > t || (key == t && i <= upto); };
  if (k < row.n) {
    unsigned long long above;
    t = radix_select(s, row, [](uint32_t, int) { return 1ull; }, (unsigned long long)k, above);
    const double ties = (double)(k - (int64_t)above);
    upto = find_id(s, [&](int i) { return row.key(i) == t ? 1.0 : 0.0; }, row.n, -1.0, ties - 1.0, ignored);
  }
  if (use_p) {
    const auto amount = [&](uint32_t key, int i) {
      return kept(key, i) ? (unsigned long long)(weight(key) * kFixed + 0.5) : 0ull;
    };
    // the whole sum: what lies above a key that none reaches
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
    const double part = (p > 0.f ? (double)p : 0.0) * (double)sum;
    const unsigned long long need = part > 1.0 ? (unsigned long long)__builtin_ceil(part) : 1ull;
    unsigned long long above;
    const uint32_t tp = radix_select(s, row, amount, need, above);
    const unsigned long long each = (unsigned long long)(weight(tp) * kFixed + 0.5);
    if (each > 0) {
      const double ties = (double)((need - above + each - 1) / each);
      upto = find_id(s, [&](int i) { return row.key(i) == tp ? 1.0 : 0.0; }, row.n, -1.0, ties - 1.0, ignored);
      t = tp;
    }
  }
  const auto share = [&](int i) {
    const uint32_t key = row.key(i);
    if (!kept(key, i)) return 0.0;
    const double w = weight(key);
    return use_min && w < (double)few ? 0.0 : w;
  };
  double total;
  const int token = find_id(s, share, row.n, (double)u, 0.0, total);
  if (tid == 0) {
    a.tokens[r] = token;
    if (a.logprobs) a.logprobs[r] = (float)log(weight(row.key(token)) / total);
  }
}

}  // namespace

size_t sample_workspace_bytes(int64_t, int64_t) { return 0; }

void launch_sample(const SampleArgs& a, void*, hipStream_t stream) {
  const dim3 grid((unsigned)a.rows);
  if (a.dtype == W4_OUT_F32) sample_kernel<float><<<grid, kSampleThreads, 0, stream>>>(a);
  else sample_kernel<uint16_t><<<grid, kSampleThreads, 0, stream>>>(a);
}

}  // namespace w4
