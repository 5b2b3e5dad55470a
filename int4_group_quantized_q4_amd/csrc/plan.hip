// The plan of a serving step over the paged cache: pages taken from and put onto
// the stack of free ones, block table columns, slots and positions of the step's
// rows, all from the sequences' lengths on the device.
//
// With have_i = ceil(len_i / p), want_i = ceil((len_i + new_i) / p) - have_i and
// the running sums W_i, R_i of want and new over the sequences, sequence i gets
// its pages and rows where W_i <= free pages and R_i <= max_rows.  Both sums
// grow, so that holds up to some sequence and for none behind it: among the
// sequences that get something, the sums of what was asked are those of what was
// given, and one scan gives the stack and row offsets.
//
// Bound by latency: one workgroup, a thread a sequence, as the stack's end and
// the scans are common to all.

#include "common.h"
#include "serving.h"

namespace w4 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

// Inclusive sums of v over the workgroup; total: that of all threads.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s_wave, int64_t& total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int64_t w = __shfl_up((long long)v, o, 64);
    if (lane >= o) v += w;
  }
  __syncthreads();   // s_wave of the scan before is read
  if (lane == 63) s_wave[wv] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const int64_t s = s_wave[w];
    if (w < wv) before += s;
    total += s;
  }
  return v + before;
}

struct Seq {
  int64_t len, fresh;   // tokens held, new ones (0 for an ended or a bad one)
  int64_t have, want;   // pages held (of an ended one: given back), pages asked
  bool ended, bad;
};

__device__ __forceinline__ Seq load_seq(const PlanArgs& a, int i) {
  Seq s{};
  if (i >= a.seqs) return s;
  s.len = a.lens[i];
  const int64_t n = a.new_tokens[i];
  s.ended = n < 0;
  s.fresh = s.ended ? 0 : n;
  s.bad = s.len < 0 || s.len + s.fresh > (a.width << a.page_shift);
  if (s.bad) {
    s.ended = false;
    s.fresh = 0;
    return s;
  }
  const int64_t up = ((int64_t)1 << a.page_shift) - 1;
  s.have = (s.len + up) >> a.page_shift;
  s.want = ((s.len + s.fresh + up) >> a.page_shift) - s.have;
  return s;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
  __shared__ int64_t s_wave[kPlanWaves];
  __shared__ unsigned long long s_cut, s_given, s_bad, s_short;
  const int tid = threadIdx.x, lane = tid & 63;
  int64_t held = a.free_count[0];
  held = held < 0 ? 0 : held > a.capacity ? a.capacity : held;
  if (tid == 0) {
    s_cut = 0;
    s_given = 0;
    s_bad = 0;
    s_short = 0;
    a.offsets[0] = 0;
  }

  // pages of ended sequences onto the stack
  int64_t back = 0;
  for (int i0 = 0; i0 < a.seqs; i0 += kPlanThreads) {
    const Seq s = load_seq(a, i0 + tid);
    const int64_t mine = s.ended ? s.have : 0;
    int64_t total;
    const int64_t at = held + back + block_scan(mine, s_wave, total) - mine;
    back += total;
    for (uint64_t todo = __ballot(mine > 0); todo; todo &= todo - 1) {
      const int l = __builtin_ctzll(todo);
      const int64_t n = __shfl((long long)mine, l, 64), to = __shfl((long long)at, l, 64);
      const int32_t* from = a.table + (int64_t)(i0 + tid - lane + l) * a.width;
      for (int64_t c = lane; c < n; c += 64)
        if (to + c < a.capacity) a.free_pages[to + c] = from[c];
    }
  }
  const int64_t lost = held + back > a.capacity ? held + back - a.capacity : 0;
  const int64_t top = held + back - lost;
  __syncthreads();   // the stack is whole

  int64_t pages = 0, rows = 0;   // asked by the sequences before
  for (int i0 = 0; i0 < a.seqs; i0 += kPlanThreads) {
    const int i = i0 + tid;
    const Seq s = load_seq(a, i);
    int64_t total_pages, total_rows;
    const int64_t upto = pages + block_scan(s.want, s_wave, total_pages);
    const int64_t row_end = rows + block_scan(s.fresh, s_wave, total_rows);
    const bool fits = i < a.seqs && upto <= top && row_end <= a.max_rows;
    pages += total_pages;
    rows += total_rows;
    if (fits) {
      atomicMax(&s_cut, (unsigned long long)row_end);
      atomicMax(&s_given, (unsigned long long)upto);
    }
    if (s.bad) atomicAdd(&s_bad, 1ull);
    if (i < a.seqs && !fits && s.fresh > 0) atomicAdd(&s_short, 1ull);
    __syncthreads();
    const int64_t cut = (int64_t)s_cut;
    if (i < a.seqs) {
      a.offsets[i + 1] = (int32_t)(fits ? row_end : cut);
      a.lens_out[i] = (int32_t)(s.ended ? 0 : fits ? s.len + s.fresh : s.len);
    }
    // new columns of the table, then the rows: a sequence's by the lanes of its wave
    const int64_t first = top - 1 - (upto - s.want);
    for (uint64_t todo = __ballot(fits && s.want > 0); todo; todo &= todo - 1) {
      const int l = __builtin_ctzll(todo);
      const int64_t n = __shfl((long long)s.want, l, 64), from = __shfl((long long)first, l, 64);
      int32_t* to = a.table + (int64_t)(i0 + tid - lane + l) * a.width + __shfl((long long)s.have, l, 64);
      for (int64_t c = lane; c < n; c += 64) to[c] = a.free_pages[from - c];
    }
    __syncthreads();   // the columns are read by other lanes
    for (uint64_t todo = __ballot(fits && s.fresh > 0); todo; todo &= todo - 1) {
      const int l = __builtin_ctzll(todo);
      const int seq = i0 + tid - lane + l;
      const int64_t n = __shfl((long long)s.fresh, l, 64), len = __shfl((long long)s.len, l, 64);
      const int64_t to = __shfl((long long)(row_end - s.fresh), l, 64);
      const int32_t* row = a.table + (int64_t)seq * a.width;
      for (int64_t c = lane; c < n; c += 64) {
        const int64_t p = len + c;
        a.slots[to + c] = ((int64_t)row[p >> a.page_shift] << a.page_shift) + (p & (((int64_t)1 << a.page_shift) - 1));
        a.positions[to + c] = (int32_t)p;
        if (a.row_seqs) a.row_seqs[to + c] = seq;
      }
    }
  }

  __syncthreads();
  const int64_t cut = (int64_t)s_cut;
  for (int64_t r = cut + tid; r < a.max_rows; r += kPlanThreads) {
    a.slots[r] = -1;
    a.positions[r] = 0;
    if (a.row_seqs) a.row_seqs[r] = -1;
  }
  if (tid == 0) {
    a.free_count_out[0] = (int32_t)(top - (int64_t)s_given);
    if (a.counters && s_bad + lost) atomicAdd(a.counters, s_bad + (unsigned long long)lost);
    if (a.counters && s_short) atomicAdd(a.counters + 1, s_short);
  }
}

}  // namespace

void launch_plan(const PlanArgs& a, hipStream_t stream) {
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
}

}  // namespace w4
