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
// the scans are common to all.  A lane writes its sequence's few pages and rows
// itself; more than that are written by the lanes of its wave together, one
// sequence after another (with all sequences taken that way, 64 of one row took 23 us for
// 7.5).  Many rows are left to a second kernel.

#include "common.h"
#include "serving.h"
#include "wave.h"

namespace w4 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kAtOnce = 8;             // pages that a lane moves at once
constexpr int kFew = 2;                // pages or rows that a lane writes for its own sequence
// Up to as many rows are written by the planning workgroup (69 rows 7.5 us in a graph, 9.0 with a second kernel; 1265
// rows of 64 sequences 11.2 and 11.1; 4000 17.2 and 11.5; 9700 29.2 and 12.7).
constexpr int kRowsHere = 1024;
constexpr int kRowThreads = 256;

// Inclusive sums of v and w over the workgroup, and their totals.
__device__ __forceinline__ void block_scan(int64_t& v, int64_t& w, int64_t (*s_wave)[2], int64_t& v_total,
                                           int64_t& w_total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  v = wave_scan(v);
  w = wave_scan(w);
  __syncthreads();   // s_wave of the scan before is read
  if (lane == 63) {
    s_wave[wv][0] = v;
    s_wave[wv][1] = w;
  }
  __syncthreads();
  v_total = w_total = 0;
#pragma unroll
  for (int i = 0; i < kPlanWaves; ++i) {
    const int64_t a = s_wave[i][0], b = s_wave[i][1];
    if (i < wv) {
      v += a;
      w += b;
    }
    v_total += a;
    w_total += b;
  }
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

__device__ __forceinline__ void store_row(const PlanArgs& a, int64_t r, const int32_t* pages, int64_t p, int seq) {
  a.slots[r] = ((int64_t)pages[p >> a.page_shift] << a.page_shift) + (p & (((int64_t)1 << a.page_shift) - 1));
  a.positions[r] = (int32_t)p;
  if (a.row_seqs) a.row_seqs[r] = seq;
}

__device__ __forceinline__ void store_pad(const PlanArgs& a, int64_t r) {
  a.slots[r] = -1;
  a.positions[r] = 0;
  if (a.row_seqs) a.row_seqs[r] = -1;
}

template <bool ROWS>   // the rows too
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
  __shared__ int64_t s_wave[kPlanWaves][2];
  __shared__ unsigned long long s_cut, s_given, s_bad, s_short;
  const int tid = threadIdx.x, lane = tid & 63;
  const Seq first = load_seq(a, tid);
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
    const Seq s = i0 == 0 ? first : load_seq(a, i0 + tid);
    const int64_t mine = s.ended ? s.have : 0;
    if (!__syncthreads_or(mine > 0)) continue;
    int64_t upto = mine, total, none = 0, none_total;
    block_scan(upto, none, s_wave, total, none_total);
    const int64_t at = held + back + upto - mine;
    back += total;
    for (uint64_t todo = __ballot(mine > 0); todo; todo &= todo - 1) {
      const int l = __builtin_ctzll(todo);
      const int64_t n = lane_value(mine, l), to = lane_value(at, l);
      const int32_t* from = a.table + (int64_t)(i0 + tid - lane + l) * a.width;
      for (int64_t c0 = lane; c0 < n; c0 += 64 * kAtOnce) {   // the loads of a round together
        int32_t page[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) page[j] = from[min(c0 + 64 * j, n - 1)];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
          if (c0 + 64 * j < n && to + c0 + 64 * j < a.capacity) a.free_pages[to + c0 + 64 * j] = page[j];
      }
    }
  }
  const int64_t lost = held + back > a.capacity ? held + back - a.capacity : 0;
  const int64_t top = held + back - lost;
  __syncthreads();   // the stack is whole

  int64_t pages = 0, rows = 0;   // asked by the sequences before
  for (int i0 = 0; i0 < a.seqs; i0 += kPlanThreads) {
    const int i = i0 + tid;
    const Seq s = i0 == 0 ? first : load_seq(a, i);
    int64_t upto = s.want, row_end = s.fresh, total_pages, total_rows;
    block_scan(upto, row_end, s_wave, total_pages, total_rows);
    upto += pages;
    row_end += rows;
    const bool fits = i < a.seqs && upto <= top && row_end <= a.max_rows;
    pages += total_pages;
    rows += total_rows;
    // the last sequence that fits has the largest sums
    const uint64_t fit = __ballot(fits);
    if (fit && lane == 63 - __builtin_clzll(fit)) {
      atomicMax(&s_cut, (unsigned long long)row_end);
      atomicMax(&s_given, (unsigned long long)upto);
    }
    const uint64_t bad = __ballot(s.bad), lacks = __ballot(i < a.seqs && !fits && s.fresh > 0);
    if (lane == 0 && bad) atomicAdd(&s_bad, (unsigned long long)__builtin_popcountll(bad));
    if (lane == 0 && lacks) atomicAdd(&s_short, (unsigned long long)__builtin_popcountll(lacks));
    // new columns of the table
    int32_t* table = a.table + (int64_t)i * a.width;
    const int64_t from = top - 1 - (upto - s.want);
    if (fits && s.want <= kFew)
      for (int64_t c = 0; c < s.want; ++c) table[s.have + c] = a.free_pages[from - c];
    for (uint64_t todo = __ballot(fits && s.want > kFew); todo; todo &= todo - 1) {
      const int l = __builtin_ctzll(todo);
      const int64_t n = lane_value(s.want, l), top_l = lane_value(from, l);
      int32_t* to = a.table + (int64_t)(i0 + tid - lane + l) * a.width + lane_value(s.have, l);
      for (int64_t c = lane; c < n; c += 64) to[c] = a.free_pages[top_l - c];
    }
    __syncthreads();   // the cut; the columns are read by other lanes
    const int64_t cut = (int64_t)s_cut;
    if (i < a.seqs) {
      a.offsets[i + 1] = (int32_t)(fits ? row_end : cut);
      a.lens_out[i] = (int32_t)(s.ended ? 0 : fits ? s.len + s.fresh : s.len);
    }
    if constexpr (ROWS) {
      if (fits && s.fresh <= kFew)
        for (int64_t c = 0; c < s.fresh; ++c) store_row(a, row_end - s.fresh + c, table, s.len + c, i);
      for (uint64_t todo = __ballot(fits && s.fresh > kFew); todo; todo &= todo - 1) {
        const int l = __builtin_ctzll(todo);
        const int seq = i0 + tid - lane + l;
        const int64_t n = lane_value(s.fresh, l), len = lane_value(s.len, l), to = lane_value(row_end, l) - n;
        for (int64_t c = lane; c < n; c += 64) store_row(a, to + c, a.table + (int64_t)seq * a.width, len + c, seq);
      }
    }
  }

  __syncthreads();
  if constexpr (ROWS)
    for (int64_t r = (int64_t)s_cut + tid; r < a.max_rows; r += kPlanThreads) store_pad(a, r);
  if (tid == 0) {
    a.free_count_out[0] = (int32_t)(top - (int64_t)s_given);
    if (a.counters && s_bad + lost) atomicAdd(a.counters, s_bad + (unsigned long long)lost);
    if (a.counters && s_short) atomicAdd(a.counters + 1, s_short);
  }
}

// A row a thread, from what plan_kernel left.
__global__ void __launch_bounds__(kRowThreads) plan_rows_kernel(PlanArgs a) {
  const int64_t r = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (r >= a.max_rows) return;
  if (a.seqs == 0 || r >= a.offsets[a.seqs]) {
    store_pad(a, r);
    return;
  }
  int lo = 0, hi = a.seqs;   // the last sequence that starts at r or before: those without rows are passed over
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.offsets[mid] <= r) lo = mid;
    else hi = mid;
  }
  store_row(a, r, a.table + (int64_t)lo * a.width, (int64_t)a.lens_out[lo] - (a.offsets[lo + 1] - r), lo);
}

}  // namespace

void launch_plan(const PlanArgs& a, hipStream_t stream) {
  if (a.max_rows <= kRowsHere) {
    plan_kernel<true><<<1, kPlanThreads, 0, stream>>>(a);
    return;
  }
  plan_kernel<false><<<1, kPlanThreads, 0, stream>>>(a);
  plan_rows_kernel<<<(unsigned)((a.max_rows + kRowThreads - 1) / kRowThreads), kRowThreads, 0, stream>>>(a);
}

}  // namespace w4
