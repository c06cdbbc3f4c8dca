// evict.hip -- eviction from the paged cache: which rows of a request are kept,
// and their move to pages of their own (gfx950).
//
// Choice: of a slot's R rows the first `first` and the last `recent` stay, and of
// those between them the ones with the greatest weights, ties to the lower row.
// The weights are ordered as 32-bit keys, and the key of the last row that is kept
// is found digit by digit.
//
// It is latency: 64 slots of 4,200 to 16,384 rows take 12.4 us in one launch (three
// histograms in LDS, the writes); a million rows of one slot 34 us in four launches of 6,
// 9, 8 and 12 (one workgroup that reads them four times took 1,348).
//
// Move: row i of a slot's list goes to row i of pages taken from the free list,
// in slot order.  Every workgroup scans all slots into LDS, as the slot map
// does, and takes its share of the rows, table entries and pages given back.
// Bound by HBM: 262,144 V41 rows of 64 slots, 280 MB, take 70 us (4.0 TB/s; more
// waves, more loads a turn and non-temporal ones measured the same or slower); 1,024
// V41_FP4 rows 5.4.
#include <algorithm>

#include "launch_evict.hpp"
#include "layout.hpp"
#include "row_ops.hpp"

namespace kvc {

namespace {

// ------------------------------------------------------------------ choice
// The key of the last row kept is found digit by digit (12, 10 and 10 bits; in
// segments 11, 11 and 10) from histograms of the candidates' keys, and the rows are
// then written in order.
//   select_registers_kernel  rows of weights of up to kSelectRegisterRows: one
//                            workgroup a slot, the keys in registers, read once
//   select_count / select_write  longer ones of up to kSelectSegmentSlots slots: a slot's
//                            rows in segments, one workgroup each; a launch a digit
//                            and one that writes.  A segment's histogram lies in
//                            the workspace, and each workgroup of the next launch
//                            adds what it needs of the slot's for itself -- no
//                            atomics in memory, nothing to clear -- together with
//                            those of the segments before its own, which say where
//                            it writes.
//   select_stream_kernel     longer ones of more slots, which fill the card with a
//                            workgroup each: the keys are read once a digit
constexpr int kSelectBlock = 1024;
constexpr int kSelectWaves = kSelectBlock / kLanes;
constexpr int kTopBits = 12, kLowBits = 10;
constexpr int kTopBins = 1 << kTopBits, kLowBins = 1 << kLowBits;
constexpr int kShift[3] = {20, 10, 0};

// Order of the weights as unsigned keys: NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.0f);
  const uint32_t k = b ^ ((int32_t)b < 0 ? 0xFFFFFFFFu : 0x80000000u);
  return w != w ? 0u : k;
}

// inclusive sum over the workgroup's threads, *total of all; buf: kSelectWaves
// words that no thread still reads
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t* buf, int32_t* total) {
  const int lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  v = wave_incl_scan_i32(v);
  if (lane == kLanes - 1) buf[wave] = v;
  __syncthreads();
  const int32_t t = wave_incl_scan_i32(lane < kSelectWaves ? buf[lane] : 0);
  *total = __builtin_amdgcn_readlane(t, kLanes - 1);
  return wave == 0 ? v : v + __builtin_amdgcn_readlane(t, wave - 1);
}

// What is decided of a slot by its length and budget alone
struct Choice {
  int32_t rows, keep;          // rows it has, rows kept (-1: inactive or refused)
  int32_t lo, hi;              // rows [lo, hi) compete for ...
  int32_t take;                // ... so many places
  bool all;                    // none does
};
__device__ __forceinline__ Choice choice_of(const SelectParams& p, int b, bool report) {
  Choice c{};
  const int32_t len = p.lens[b];
  c.keep = -1;
  c.all = true;
  if (len < 0) return c;
  c.rows = len >> (p.ratio - 1);
  if (c.rows > p.w_width) {
    if (report && threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, kStPtRange);
    return c;
  }
  int32_t budget = p.budgets != nullptr ? p.budgets[b] : p.budget;
  if (budget < 0 || budget > p.kept_width) budget = p.kept_width;
  c.keep = min(c.rows, budget);
  if (c.rows <= budget) return c;
  c.lo = min(p.first, budget);
  const int32_t recent = min(p.recent, budget - c.lo);
  c.hi = c.rows - recent;
  c.take = budget - c.lo - recent;
  c.all = c.take == 0;
  return c;
}

// A slot's lists and what of them does not depend on the weights: the count, the
// rows that stay whatever theirs, and what follows the list.  The slot's
// workgroups, `of` of them, take a share each.
struct Lists {
  const float* w;
  int32_t* kept;
  float* kw;
  __device__ __forceinline__ Lists(const SelectParams& p, int64_t b)
      : w(p.weights + b * p.w_stride), kept(p.kept + b * p.kept_stride),
        kw(p.kept_weights != nullptr ? p.kept_weights + b * p.kw_stride : nullptr) {}
  __device__ __forceinline__ void put(int32_t i, int32_t r, float v) const {
    kept[i] = r;
    if (kw != nullptr) kw[i] = v;
  }
  __device__ __forceinline__ void begin(const SelectParams& p, int b, const Choice& c, int part, int of) const {
    if (threadIdx.x == 0 && part == 0) p.counts[b] = c.keep;
    // (all rows kept: lo and take are 0 or the first rows and none, and row i is i
    // up to lo, then counted from the end)
    const bool whole = c.keep == c.rows;
    for (int64_t i = part * kSelectBlock + threadIdx.x; i < p.kept_width; i += of * kSelectBlock) {
      if (i >= c.lo && i < c.lo + c.take) continue;
      const int32_t r = i >= c.keep ? -1 : whole || i < c.lo ? (int32_t)i : c.rows - (c.keep - (int32_t)i);
      put((int32_t)i, r, r >= 0 ? w[r] : 0.0f);
    }
  }
};

// Of N bins a thread, n[k] keys in the k-th from the greatest down (thread 0 has
// the greatest): the bin that holds the left-th greatest key, and which of that
// bin's it is.  found: 2 words that no thread still reads.
struct Digit {
  uint32_t bin;
  int32_t left;
};
template <int N>
__device__ __forceinline__ Digit find_digit(const int32_t (&n)[N], int32_t left, int32_t* buf, int32_t* found) {
  int32_t sum = 0, total;
#pragma unroll
  for (int k = 0; k < N; ++k) sum += n[k];
  int32_t above = block_scan(sum, buf, &total) - sum;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (above < left && above + n[k] >= left) {
      found[0] = N * kSelectBlock - 1 - N * (int)threadIdx.x - k;
      found[1] = left - above;
    }
    above += n[k];
  }
  __syncthreads();
  return Digit{(uint32_t)found[0], found[1]};
}
template <int N>
__device__ __forceinline__ void bins_of(const uint32_t* hist, int32_t (&n)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) n[k] = (int32_t)hist[N * kSelectBlock - 1 - N * (int)threadIdx.x - k];
}

// lanes below this one in m
__device__ __forceinline__ int32_t lanes_before(uint64_t m) {
  return (int32_t)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// Writes the kept ones of 64 rows, a lane each, and moves the counts past them.
// key: of the last row kept, of whose equals the first `left` are kept.
struct Written {
  int32_t above, equal;        // rows before these that are greater, equal
};
__device__ __forceinline__ void write_rows(const Lists& l, const Choice& c, Written& at, uint32_t key, int32_t left,
                                           int32_t r, float v, bool in) {
  const uint32_t k = weight_key(v);
  const uint64_t gt = __ballot(in && k > key), eq = __ballot(in && k == key);
  const int32_t g = at.above + lanes_before(gt), e = at.equal + lanes_before(eq);
  if (in && (k > key || (k == key && e < left))) l.put(c.lo + g + min(e, left), r, v);
  at.above += __builtin_popcountll(gt);
  at.equal += __builtin_popcountll(eq);
}

// E * 64 rows a wave
template <int E>
__global__ __launch_bounds__(kSelectBlock) void select_registers_kernel(SelectParams p) {
  __shared__ uint32_t hist[kTopBins];
  __shared__ int32_t buf[2][kSelectWaves], found[3][2];
  __shared__ int32_t counts[kSelectWaves][2];
  const int b = blockIdx.x, tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
  const Choice c = choice_of(p, b, true);
  const Lists l(p, b);
  const int32_t r0 = c.lo + wave * E * kLanes + lane;
  float v[E];
  if (!c.all) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = r0 + i * kLanes < c.hi ? l.w[r0 + i * kLanes] : 0.0f;
  }
  l.begin(p, b, c, 0, 1);
  if (c.all) return;
  Digit d{0, c.take};
  uint32_t key = 0;
  // (32 keys are made from the weights wherever they are needed: both would not fit, and
  // the spills cost more -- 512 slots 62 us for 57; with 16 they fit, 13 us for 15)
  auto keep_weights = [&]() {
    if constexpr (E <= 24) return;
#pragma unroll
    for (int i = 0; i < E; ++i) asm volatile("" : "+v"(v[i]));
  };
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    keep_weights();
    for (int i = tid; i < (pass == 0 ? kTopBins : kLowBins); i += kSelectBlock) hist[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const uint32_t k = weight_key(v[i]);
      if (r0 + i * kLanes < c.hi && (pass == 0 || k >> (kShift[pass] + kLowBits) == key))
        atomicAdd(&hist[pass == 0 ? k >> kShift[0] : k >> kShift[pass] & (kLowBins - 1)], 1u);
    }
    __syncthreads();
    if (pass == 0) {
      int32_t n[kTopBins / kSelectBlock];
      bins_of(hist, n);
      d = find_digit(n, d.left, buf[0], found[0]);
      key = d.bin;
    } else {
      int32_t n[1];
      bins_of(hist, n);
      d = find_digit(n, d.left, buf[pass & 1], found[pass]);
      key = key << kLowBits | d.bin;
    }
  }
  Written at{0, 0};
  keep_weights();
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t k = weight_key(v[i]);
    const bool in = r0 + i * kLanes < c.hi;
    at.above += __builtin_popcountll(__ballot(in && k > key));
    at.equal += __builtin_popcountll(__ballot(in && k == key));
  }
  if (lane == 0) counts[wave][0] = at.above, counts[wave][1] = at.equal;
  __syncthreads();
  at = Written{0, 0};
  for (int w = 0; w < kSelectWaves; ++w) {
    if (w < wave) at.above += counts[w][0], at.equal += counts[w][1];
  }
  keep_weights();
#pragma unroll
  for (int i = 0; i < E; ++i)
    write_rows(l, c, at, key, d.left, r0 + i * kLanes, v[i], r0 + i * kLanes < c.hi);
}

__global__ __launch_bounds__(kSelectBlock) void select_stream_kernel(SelectParams p) {
  __shared__ uint32_t hist[kTopBins];
  __shared__ int32_t buf[2][kSelectWaves], found[3][2];
  const int b = blockIdx.x, tid = threadIdx.x;
  const Choice c = choice_of(p, b, true);
  const Lists l(p, b);
  l.begin(p, b, c, 0, 1);
  if (c.all) return;
  Digit d{0, c.take};
  uint32_t key = 0;
  for (int pass = 0; pass < 3; ++pass) {
    for (int i = tid; i < (pass == 0 ? kTopBins : kLowBins); i += kSelectBlock) hist[i] = 0;
    __syncthreads();
    for (int64_t r = (int64_t)c.lo + tid; r < c.hi; r += kSelectBlock) {
      const uint32_t k = weight_key(l.w[r]);
      if (pass == 0) atomicAdd(&hist[k >> kShift[0]], 1u);
      else if (k >> (kShift[pass] + kLowBits) == key) atomicAdd(&hist[k >> kShift[pass] & (kLowBins - 1)], 1u);
    }
    __syncthreads();
    if (pass == 0) {
      int32_t n[kTopBins / kSelectBlock];
      bins_of(hist, n);
      d = find_digit(n, d.left, buf[0], found[0]);
      key = d.bin;
    } else {
      int32_t n[1];
      bins_of(hist, n);
      d = find_digit(n, d.left, buf[pass & 1], found[pass]);
      key = key << kLowBits | d.bin;
    }
  }
  int32_t above = 0, equal = 0;               // of the rows before this turn's
  int turn = 0;
  for (int64_t t0 = c.lo; t0 < c.hi; t0 += kSelectBlock, turn ^= 1) {
    const int64_t r = t0 + tid;
    const float v = r < c.hi ? l.w[r] : 0.0f;
    const uint32_t k = weight_key(v);
    const bool gt = r < c.hi && k > key, eq = r < c.hi && k == key;
    int32_t total;
    // (both counts of a turn fit 16 bits)
    const int32_t end = block_scan((gt ? 1 : 0) | (eq ? 1 << 16 : 0), buf[turn], &total);
    const int32_t g = above + (end & 0xFFFF) - (gt ? 1 : 0), e = equal + (end >> 16) - (eq ? 1 : 0);
    if (gt || (eq && e < d.left)) l.put(c.lo + g + min(e, d.left), (int32_t)r, v);
    above += total & 0xFFFF;
    equal += total >> 16;
  }
}

// ---- segments
constexpr int kSegBits[3] = {11, 11, 10}, kSegShift[3] = {21, 10, 0};
constexpr int kCoarse = 64;                   // a histogram's sums of so many equal stretches lie in front of it
static_assert(kSelectWords == kCoarse + (1 << kSegBits[0]) && kSegBits[1] <= kSegBits[0] && kSegBits[2] <= kSegBits[0],
              "words of a histogram");
constexpr int kTurn = 16;                     // rows a thread has in registers

// A segment of a slot: what is known of the key, and of the segments before it
struct Found {
  uint32_t key;                // digits found, the last in the low bits
  int32_t left;                // of the rows with them, so many are kept
  Written before;              // in the segments before this one: rows kept for certain, rows with all digits
};

// Sums over the segments' counts, a lane each: all of them, and those of segments before
// this one.  Every wave has them.
struct Sums {
  int32_t all, before;
};
struct SumsBuf {
  int32_t all[kSelectWaves][kLanes], before[kSelectWaves][kLanes];
};
// W lanes of counts at `at` of each segment's words; lanes past W get 0
template <int W>
__device__ __forceinline__ Sums sum_segments(const SelectParams& p, const uint32_t* at, int s, SumsBuf& buf) {
  constexpr int G = kLanes / W;                // segments a wave reads at once
  const int lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  Sums v{0, 0};
#pragma unroll 8
  for (int t = wave * G + lane / W; t < p.segments; t += kSelectWaves * G) {
    const int32_t n = (int32_t)at[(int64_t)t * kSelectWords + lane % W];
    v.all += n;
    v.before += t < s ? n : 0;
  }
#pragma unroll
  for (int d = W; d < kLanes; d <<= 1) {
    v.all += __shfl_xor(v.all, d);
    v.before += __shfl_xor(v.before, d);
  }
  buf.all[wave][lane] = v.all;
  buf.before[wave][lane] = v.before;
  __syncthreads();
  v = Sums{0, 0};
  // (of the waves that had any)
  const int waves = min(kSelectWaves, (p.segments + G - 1) / G);
#pragma unroll 4
  for (int w = 0; w < waves; ++w) v.all += buf.all[w][lane], v.before += buf.before[w][lane];
  return lane < W ? v : Sums{0, 0};
}

// The lane (greatest first) whose counts hold the left-th key, which of that lane's it
// is, and the counts before this segment in greater lanes and in that one
struct LaneFound {
  int32_t lane, left;
  Written before;
};
__device__ __forceinline__ LaneFound find_lane(const Sums& v, int32_t left) {
  const int32_t above = __builtin_amdgcn_readlane(wave_incl_scan_i32(v.all), kLanes - 1) - wave_incl_scan_i32(v.all);
  const int32_t end = wave_incl_scan_i32(v.before);
  const uint64_t hit = __ballot(above < left && above + v.all >= left);
  const int lane = __builtin_ctzll(hit | 1ull << 63);   // (a lane, also if the counts were another call's)
  return LaneFound{lane, left - __builtin_amdgcn_readlane(above, lane),
                   {__builtin_amdgcn_readlane(end, kLanes - 1) - __builtin_amdgcn_readlane(end, lane),
                    __builtin_amdgcn_readlane(v.before, lane)}};
}

// The digit that the histograms of the last launch give, from the slot's sums: first of
// their stretches, then of the bins of the one that holds it (24 KB a workgroup for
// 64 segments, where the whole histograms are 512: a million rows took 44 us with them)
template <int BINS>
__device__ __forceinline__ Found next_digit(const SelectParams& p, Found f, const uint32_t* hists, int s, SumsBuf (&buf)[2]) {
  constexpr int W = BINS / kCoarse;
  const LaneFound c = find_lane(sum_segments<kCoarse>(p, hists, s, buf[0]), f.left);
  const LaneFound d = find_lane(sum_segments<W>(p, hists + kCoarse + c.lane * W, s, buf[1]), c.left);
  f.key = f.key * BINS + (uint32_t)(c.lane * W + d.lane);
  f.left = d.left;
  f.before.above += c.before.above + d.before.above;
  f.before.equal = d.before.equal;
  return f;
}

__device__ __forceinline__ uint32_t* hists_of(const SelectParams& p, int pass, int64_t seg) {
  return p.hists + ((int64_t)pass * p.num_slots * p.segments + seg) * kSelectWords;
}

// Counts the segment's keys that begin with the PASS digits found -- the last of them
// found here -- by their next one.
template <int PASS>
__global__ __launch_bounds__(kSelectBlock) void select_count_kernel(SelectParams p) {
  constexpr int BINS = 1 << kSegBits[PASS];
  __shared__ uint32_t hist[BINS];
  __shared__ SumsBuf buf[2];
  const int s = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const Choice c = choice_of(p, b, PASS == 0 && s == 0);
  const Lists l(p, b);
  const int64_t seg = (int64_t)b * p.segments + s;
  const int64_t begin = c.lo + s * p.segment_rows, end = min((int64_t)c.hi, begin + p.segment_rows);
  // (asked for before the digit is known)
  float v[kTurn];
#pragma unroll
  for (int i = 0; i < kTurn; ++i) v[i] = begin + tid + i * kSelectBlock < end ? l.w[begin + tid + i * kSelectBlock] : 0.0f;
  for (int i = tid; i < BINS; i += kSelectBlock) hist[i] = 0;
  if (PASS == 0) l.begin(p, b, c, s, p.segments);
  if (c.all) return;
  Found f{0, c.take, {0, 0}};
  if constexpr (PASS == 2) {
    const int32_t* st = p.states + 4 * seg;
    f = Found{(uint32_t)st[0], st[1], {st[2], 0}};
  }
  if constexpr (PASS > 0)
    f = next_digit<1 << kSegBits[PASS - 1]>(p, f, hists_of(p, PASS - 1, (int64_t)b * p.segments), s, buf);
  __syncthreads();
  auto count = [&](float w, bool in) {
    const uint32_t k = weight_key(w);
    const uint64_t up = (uint64_t)k >> (kSegShift[PASS] + kSegBits[PASS]);
    if (in && up == f.key) atomicAdd(&hist[k >> kSegShift[PASS] & (BINS - 1)], 1u);
  };
#pragma unroll
  for (int i = 0; i < kTurn; ++i) count(v[i], begin + tid + i * kSelectBlock < end);
  for (int64_t r = begin + tid + kTurn * kSelectBlock; r < end; r += kSelectBlock) count(l.w[r], true);
  __syncthreads();
  uint32_t* out = hists_of(p, PASS, seg);
  constexpr int W = BINS / kCoarse;
#pragma unroll
  for (int i = tid; i < BINS; i += kSelectBlock) {
    int32_t n = (int32_t)hist[i];
    out[kCoarse + i] = (uint32_t)n;
#pragma unroll
    for (int d = 1; d < W; d <<= 1) n += __shfl_xor(n, d);
    if (tid % W == 0) out[i / W] = (uint32_t)n;
  }
  if (PASS > 0 && tid == 0) {
    int32_t* st = p.states + 4 * seg;
    st[0] = (int32_t)f.key, st[1] = f.left, st[2] = f.before.above;
  }
}

__global__ __launch_bounds__(kSelectBlock) void select_write_kernel(SelectParams p) {
  __shared__ SumsBuf buf[2];
  __shared__ int32_t counts[2][kSelectWaves][2];
  const int s = blockIdx.x, b = blockIdx.y, lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  const Choice c = choice_of(p, b, false);
  if (c.all) return;
  const Lists l(p, b);
  const int64_t seg = (int64_t)b * p.segments + s;
  const int64_t begin = c.lo + s * p.segment_rows, end = min((int64_t)c.hi, begin + p.segment_rows);
  // turns of 16 waves of 1,024 rows
  float v[kTurn];
  int64_t r0 = begin + wave * kTurn * kLanes + lane;
  auto fetch = [&]() {
#pragma unroll
    for (int i = 0; i < kTurn; ++i) v[i] = r0 + i * kLanes < end ? l.w[r0 + i * kLanes] : 0.0f;
  };
  fetch();
  const int32_t* st = p.states + 4 * seg;
  Found f{(uint32_t)st[0], st[1], {st[2], 0}};
  f = next_digit<1 << kSegBits[2]>(p, f, hists_of(p, 2, (int64_t)b * p.segments), s, buf);
  int turn = 0;
  for (int64_t t0 = begin; t0 < end; t0 += kSelectBlock * kTurn, turn ^= 1) {
    if (t0 > begin) {
      r0 += kSelectBlock * kTurn;
      fetch();
    }
    Written at{0, 0};
#pragma unroll
    for (int i = 0; i < kTurn; ++i) {
      const uint32_t k = weight_key(v[i]);
      const bool in = r0 + i * kLanes < end;
      at.above += __builtin_popcountll(__ballot(in && k > f.key));
      at.equal += __builtin_popcountll(__ballot(in && k == f.key));
    }
    if (lane == 0) counts[turn][wave][0] = at.above, counts[turn][wave][1] = at.equal;
    __syncthreads();
    const int32_t above = wave_incl_scan_i32(lane < kSelectWaves ? counts[turn][lane][0] : 0);
    const int32_t equal = wave_incl_scan_i32(lane < kSelectWaves ? counts[turn][lane][1] : 0);
    at = f.before;
    if (wave > 0) {
      at.above += __builtin_amdgcn_readlane(above, wave - 1);
      at.equal += __builtin_amdgcn_readlane(equal, wave - 1);
    }
    f.before.above += __builtin_amdgcn_readlane(above, kLanes - 1);
    f.before.equal += __builtin_amdgcn_readlane(equal, kLanes - 1);
#pragma unroll
    for (int i = 0; i < kTurn; ++i)
      write_rows(l, c, at, f.key, f.left, (int32_t)(r0 + i * kLanes), v[i], r0 + i * kLanes < end);
  }
}

// ------------------------------------------------------------------ move
constexpr int kCompactBlock = 512;
constexpr int kCompactWaves = kCompactBlock / kLanes;
constexpr int kCompactGrid = 512;
constexpr int kBatch = 32;       // rows a wave moves at once
constexpr int kEntries = 256;    // table entries a wave writes at once

// Sums over slots saturate (a batch may ask for more than there can be before
// it is refused)
constexpr uint32_t kSat = 0x7FFFFFFF;
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }
__device__ __forceinline__ uint32_t wave_sat_scan(uint32_t v) {
  v = sat_add(v, (uint32_t)dpp_shr_or_zero<0x111>((int32_t)v));
  v = sat_add(v, (uint32_t)dpp_shr_or_zero<0x112>((int32_t)v));
  v = sat_add(v, (uint32_t)dpp_shr_or_zero<0x114>((int32_t)v));
  v = sat_add(v, (uint32_t)dpp_shr_or_zero<0x118>((int32_t)v));
  v = sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowBcast15, 0xA, 0xF, false));
  return sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowBcast31, 0xC, 0xF, false));
}
// inclusive saturating sum over the workgroup's threads, *total of all; buf:
// kCompactWaves words that no thread still reads
__device__ __forceinline__ uint32_t block_sat_scan(uint32_t v, uint32_t* buf, uint32_t* total) {
  const int lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  v = wave_sat_scan(v);
  if (lane == kLanes - 1) buf[wave] = v;
  __syncthreads();
  const uint32_t t = wave_sat_scan(lane < kCompactWaves ? buf[lane] : 0u);
  *total = (uint32_t)__builtin_amdgcn_readlane((int)t, kLanes - 1);
  return wave == 0 ? v : sat_add(v, (uint32_t)__builtin_amdgcn_readlane((int)t, wave - 1));
}

// What one slot asks for, before the shared limits are looked at
struct Move {
  int32_t len, rows;           // tokens (as given), cached rows
  int32_t count;               // rows kept
  int32_t take, give;          // pages, 0 for a slot that stays as it is
  bool wants, ok;              // has rows to drop; and its table and list hold them
};
__device__ __forceinline__ Move move_of(const CompactParams& p, int b, int32_t* bad) {
  Move m{};
  m.len = p.lens[b];
  m.rows = m.len >= 0 ? m.len >> (p.ratio - 1) : 0;
  m.count = p.counts[b];
  m.wants = m.count >= 0 && m.count < m.rows;
  if (!m.wants) return m;
  const int64_t ps = int64_t(1) << p.cache.page_bits;
  const int64_t give = (m.rows + ps - 1) >> p.cache.page_bits;
  m.ok = give <= p.pt_width && m.count <= p.kept_width && (p.weights == nullptr || m.count <= p.w_width);
  if (!m.ok) {
    *bad |= kStPtRange;
    return m;
  }
  m.give = (int32_t)give;
  m.take = (int32_t)((m.count + ps - 1) >> p.cache.page_bits);
  return m;
}

// 16-byte units of a row, the scale part last (V4: one of 8 bytes)
template <int L>
struct RowUnits {
  static constexpr int kData = LayoutTraits<L>::kData / 16;
  static constexpr int kAll = kData + (LayoutTraits<L>::kScale + 15) / 16;
  // byte of unit k in a page whose data parts take `all_data` bytes
  static __device__ __forceinline__ uint32_t at(int k, uint32_t row, uint32_t all_data) {
    return k < kData ? row * LayoutTraits<L>::kData + 16 * k
                     : all_data + row * LayoutTraits<L>::kScale + 16 * (k - kData);
  }
  static __device__ __forceinline__ u32x4 load(const uint8_t* a, int k) {
    if (L == kV4 && k == kData) {
      const u32x2 v = *(const u32x2*)a;
      return u32x4{v.x, v.y, 0u, 0u};
    }
    return *(const u32x4*)a;
  }
  static __device__ __forceinline__ void store(uint8_t* a, int k, u32x4 v) {
    if (L == kV4 && k == kData) *(u32x2*)a = u32x2{v.x, v.y};
    else *(u32x4*)a = v;
  }
};

template <int L, int SLOTS>
__global__ __launch_bounds__(kCompactBlock) void compact_kernel(CompactParams p) {
  // of each slot: the first of its rows among those moved, its place in the free
  // list, its place in the list of pages given back (-1: the slot stays as it is)
  __shared__ int32_t row0[SLOTS], take0[SLOTS], give0[SLOTS];
  __shared__ uint32_t buf[3][kCompactWaves];
  __shared__ int64_t src_page[kCompactWaves][kBatch], dst_page[kCompactWaves][kBatch];
  __shared__ uint32_t src_row[kCompactWaves][kBatch], dst_row[kCompactWaves][kBatch];
  __shared__ unsigned long long dropped;
  __shared__ int32_t refused;
  const int S = p.num_slots, tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
  const int pb = p.cache.page_bits, rl = p.ratio - 1;
  int32_t bad = 0;
  uint32_t rows_at = 0, take_at = 0, give_at = 0;
  uint32_t taken = 0, given = 0;              // of the slots that are moved, so far
  if (tid == 0) dropped = 0, refused = 0;
  // pages past the cache's own number (page 0 apart) cannot all be free
  const uint32_t n_free = (uint32_t)min(p.n_free, p.cache.num_pages - 1);
  for (int b0 = 0; b0 < S; b0 += kCompactBlock) {
    const int b = b0 + tid;
    Move m{};
    if (b < S) m = move_of(p, b, &bad);
    uint32_t total;
    const uint32_t te = sat_add(block_sat_scan((uint32_t)m.take, buf[0], &total), take_at);
    take_at = sat_add(take_at, total);
    const uint32_t ge = sat_add(block_sat_scan((uint32_t)m.give, buf[1], &total), give_at);
    give_at = sat_add(give_at, total);
    // (behind a slot refused here every one with rows to drop is: its sums are no
    // less; so the places of those that are not count no refused one)
    const bool fits = te <= n_free && (p.freed == nullptr || ge <= (uint32_t)p.freed_cap);
    const bool moved = m.ok && fits;
    if (m.ok && !fits) bad |= kStNoPage;
    const uint32_t re = sat_add(block_sat_scan(moved ? (uint32_t)m.count : 0u, buf[2], &total), rows_at);
    rows_at = sat_add(rows_at, total);
    if (b < S) {
      row0[b] = (int32_t)re - (moved ? m.count : 0);
      take0[b] = (int32_t)te - m.take;
      give0[b] = moved ? (int32_t)ge - m.give : -1;
      if (moved) taken = te, given = ge;
    }
    if (blockIdx.x == 0) {
      if (moved) atomicAdd(&dropped, (unsigned long long)(m.rows - m.count));
      if (m.wants && !moved) atomicAdd(&refused, 1);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (bad != 0 && p.status != nullptr) atomicOr(p.status, bad);
    if (p.totals != nullptr) {
      // the greatest places reached
      for (int d = kLanes / 2; d > 0; d >>= 1) {
        taken = max(taken, (uint32_t)__shfl_xor((int)taken, d));
        given = max(given, (uint32_t)__shfl_xor((int)given, d));
      }
      if (lane == 0) buf[0][wave] = taken, buf[1][wave] = given;
      __syncthreads();
      if (tid == 0) {
        for (int w = 1; w < kCompactWaves; ++w) taken = max(taken, buf[0][w]), given = max(given, buf[1][w]);
        p.totals[0] = (int32_t)taken;
        p.totals[1] = (int32_t)given;
        p.totals[2] = (int32_t)min(dropped, (unsigned long long)kSat);
        p.totals[3] = refused;
      }
    }
  }

  // rows
  const uint32_t all_data = (uint32_t)LayoutTraits<L>::kData << pb;
  const int32_t in_page = (1 << pb) - 1;
  const uint32_t wave0 = blockIdx.x * kCompactWaves + wave, waves = gridDim.x * kCompactWaves;
  // Few rows are spread over more waves.  Measured in batches of 8 and 32, us: 4,096 rows
  // of 8 slots 11.9 and 14.3, 102,400 of 200 slots 28.1 and 22.7, 262,144 of 64 slots 75.4
  // and 71.7.
  const uint32_t batch = rows_at >= (uint32_t)kBatch * kCompactGrid * kCompactWaves / 2 ? kBatch : 8;
  const uint32_t batches = (rows_at + batch - 1) / batch;
  for (uint32_t g = wave0; g < batches; g += waves) {
    const uint32_t n = min(batch, rows_at - g * batch);
    if ((uint32_t)lane < n) {
      const int32_t x = (int32_t)(g * batch) + lane;
      int lo = 0, hi = S - 1;                 // last slot with row0 <= x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (row0[mid] <= x) lo = mid;
        else hi = mid - 1;
      }
      const int64_t b = lo;
      const int32_t i = x - row0[lo];
      const int32_t id = p.kept[b * p.kept_stride + i];
      const int32_t to = p.free_pages[take0[lo] + (i >> pb)];
      if (p.weights != nullptr) p.weights[b * p.w_stride + i] = p.kept_weights[b * p.kw_stride + i];
      int64_t src = -1, dst = -1;             // (bytes; a row that cannot be read is 0)
      int32_t wrong = 0;
      if (id < 0 || id >= p.lens[b] >> rl) {
        wrong |= kStIdRange;
      } else {
        const int32_t page = p.page_table[b * p.pt_stride + (id >> pb)];
        if (page < 0 || page >= p.cache.num_pages) wrong |= kStPageRange;
        else src = page * p.cache.page_stride;
      }
      if (to < 1 || to >= p.cache.num_pages) wrong |= kStPageRange;
      else dst = to * p.cache.page_stride;
      if (wrong != 0 && p.status != nullptr) atomicOr(p.status, wrong);
      src_page[wave][lane] = src;
      dst_page[wave][lane] = dst;
      src_row[wave][lane] = (uint32_t)(id & in_page);
      dst_row[wave][lane] = (uint32_t)(i & in_page);
    }
    __builtin_amdgcn_wave_barrier();
    constexpr int U = RowUnits<L>::kAll, N = 4;
    const uint32_t units = n * U;
    for (uint32_t u0 = 0; u0 < units; u0 += N * kLanes) {
      u32x4 v[N];
      uint8_t* at[N];
      int k[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t u = u0 + j * kLanes + lane;
        at[j] = nullptr;
        v[j] = u32x4{0, 0, 0, 0};
        if (u < units) {
          const uint32_t row = u / U;
          k[j] = (int)(u - row * U);
          const int64_t src = src_page[wave][row], dst = dst_page[wave][row];
          if (src >= 0)
            v[j] = RowUnits<L>::load(p.cache.base + src + RowUnits<L>::at(k[j], src_row[wave][row], all_data), k[j]);
          if (dst >= 0) at[j] = p.cache.base + dst + RowUnits<L>::at(k[j], dst_row[wave][row], all_data);
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (at[j] != nullptr) RowUnits<L>::store(at[j], k[j], v[j]);
    }
    __builtin_amdgcn_wave_barrier();
  }

  // tables, lengths, pages given back
  const uint32_t pieces = (uint32_t)((p.pt_width + kEntries - 1) / kEntries);
  const uint64_t items = (uint64_t)pieces * (uint32_t)S;
  for (uint64_t it = wave0; it < items; it += waves) {
    const int64_t b = (int64_t)(it / pieces);
    const int64_t e0 = (int64_t)(it - (uint64_t)b * pieces) * kEntries;
    const int32_t len = p.lens[b], count = p.counts[b], back = give0[b];
    const int64_t ps = int64_t(1) << pb;
    const int64_t held = len >= 0 ? ((len >> rl) + ps - 1) >> pb : 0;
    const int64_t take = (count + ps - 1) >> pb;
    if (e0 == 0 && lane == 0) p.new_lens[b] = back >= 0 ? (count << rl) + (len & rl) : len;
    for (int64_t e = e0 + lane; e < e0 + kEntries && e < p.pt_width; e += kLanes) {
      const int32_t old = e < held ? p.page_table[b * p.pt_stride + e] : 0;
      int32_t entry = old;
      if (back >= 0) {
        entry = e < take ? p.free_pages[take0[b] + e] : 0;
        if (e < held && p.freed != nullptr) p.freed[back + e] = old;
      }
      p.new_table[b * p.nt_stride + e] = entry;
    }
  }
}

template <int L>
void launch_compact_as(const CompactParams& p, hipStream_t stream) {
  // the rows are counted on the device: as many waves as there can be rows and
  // table pieces, no more than fill the card
  const int64_t rows = (int64_t)p.num_slots * p.kept_width;
  const int64_t pieces = (p.pt_width + kEntries - 1) / kEntries * p.num_slots;
  const int64_t waves = rows / 8 + pieces + 1;
  const dim3 grid((uint32_t)std::min<int64_t>(kCompactGrid, (waves + kCompactWaves - 1) / kCompactWaves));
  if (p.num_slots <= 1024) compact_kernel<L, 1024><<<grid, kCompactBlock, 0, stream>>>(p);
  else compact_kernel<L, kMaxSlots + 1><<<grid, kCompactBlock, 0, stream>>>(p);
}

}  // namespace

hipError_t launch_select(const SelectParams& p, hipStream_t stream) {
  const dim3 slots((uint32_t)p.num_slots);
  if (p.segments > 0) {
    const dim3 grid((uint32_t)p.segments, (uint32_t)p.num_slots);
    select_count_kernel<0><<<grid, kSelectBlock, 0, stream>>>(p);
    select_count_kernel<1><<<grid, kSelectBlock, 0, stream>>>(p);
    select_count_kernel<2><<<grid, kSelectBlock, 0, stream>>>(p);
    select_write_kernel<<<grid, kSelectBlock, 0, stream>>>(p);
  } else if (p.w_width <= kSelectBlock) {
    select_registers_kernel<1><<<slots, kSelectBlock, 0, stream>>>(p);
  } else if (p.w_width <= 4 * kSelectBlock) {
    select_registers_kernel<4><<<slots, kSelectBlock, 0, stream>>>(p);
  } else if (p.w_width <= 16 * kSelectBlock) {
    select_registers_kernel<16><<<slots, kSelectBlock, 0, stream>>>(p);
  } else if (p.w_width <= 24 * kSelectBlock) {
    select_registers_kernel<24><<<slots, kSelectBlock, 0, stream>>>(p);
  } else if (p.w_width <= kSelectRegisterRows) {
    select_registers_kernel<kSelectRegisterRows / kSelectBlock><<<slots, kSelectBlock, 0, stream>>>(p);
  } else {
    select_stream_kernel<<<slots, kSelectBlock, 0, stream>>>(p);
  }
  return hipGetLastError();
}

hipError_t launch_compact(const CompactParams& p, hipStream_t stream) {
  switch (p.cache.layout) {
    case kV4: launch_compact_as<kV4>(p, stream); break;
    case kV41: launch_compact_as<kV41>(p, stream); break;
    default: launch_compact_as<kV41Fp4>(p, stream); break;
  }
  return hipGetLastError();
}

}  // namespace kvc
