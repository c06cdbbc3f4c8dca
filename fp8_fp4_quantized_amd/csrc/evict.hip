// evict.hip -- eviction from the paged cache: which rows of a request are kept,
// and their move to pages of their own (gfx950).
//
// Choice: of a slot's R rows the first `first` and the last `recent` stay, and of
// those between them the ones with the greatest weights, ties to the lower row.
// The weights are ordered as 32-bit keys; three passes over them count the
// keys' digits (11, 11 and 10 bits) and leave the key of the last row that is
// kept, a fourth writes the rows in order.  One workgroup a slot.
//
// Move: row i of a slot's list goes to row i of pages taken from the free list,
// in slot order.  Every workgroup scans all slots into LDS, as the slot map
// does, and takes its share of the rows, table entries and pages given back.
#include <algorithm>

#include "launch_evict.hpp"
#include "layout.hpp"
#include "row_ops.hpp"

namespace kvc {

namespace {

constexpr int kSelectBlock = 1024;
constexpr int kSelectWaves = kSelectBlock / kLanes;
constexpr int kBins = 2048;

// Order of the weights as unsigned keys: NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.0f);
  const uint32_t k = b ^ ((int32_t)b < 0 ? 0xFFFFFFFFu : 0x80000000u);
  return w != w ? 0u : k;
}

// inclusive sum over the workgroup's threads, *total of all; buf: kSelectWaves
// words that no thread still reads, and none may write before the next barrier
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
};
__device__ __forceinline__ Choice choice_of(const SelectParams& p, int b) {
  Choice c{};
  const int32_t len = p.lens[b];
  c.keep = -1;
  if (len < 0) return c;
  c.rows = len >> (p.ratio - 1);
  if (c.rows > p.w_width) {
    if (threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, kStPtRange);
    return c;
  }
  int32_t budget = p.budgets != nullptr ? p.budgets[b] : p.budget;
  if (budget < 0 || budget > p.kept_width) budget = p.kept_width;
  if (c.rows <= budget) {                     // every row stays
    c.keep = c.rows;
    return c;
  }
  c.keep = budget;
  c.lo = min(p.first, budget);
  const int32_t recent = min(p.recent, budget - c.lo);
  c.hi = c.rows - recent;
  c.take = budget - c.lo - recent;
  return c;
}

__global__ __launch_bounds__(kSelectBlock) void select_kernel(SelectParams p) {
  __shared__ uint32_t hist[kBins];
  __shared__ int32_t buf[2][kSelectWaves];
  __shared__ int32_t found[2];                // digit, places left for it
  const int b = blockIdx.x, tid = threadIdx.x;
  const Choice c = choice_of(p, b);
  const float* w = p.weights + b * p.w_stride;
  int32_t* kept = p.kept + b * p.kept_stride;
  float* kw = p.kept_weights != nullptr ? p.kept_weights + b * p.kw_stride : nullptr;
  const bool all = c.keep < 0 || c.keep == c.rows;
  if (tid == 0) p.counts[b] = c.keep;
  // rows kept whatever their weight, and what follows the list
  for (int32_t i = tid; i < p.kept_width; i += kSelectBlock) {
    const bool mid = !all && i >= c.lo && i < c.lo + c.take;
    if (mid) continue;
    const int32_t r = i >= c.keep ? -1 : all || i < c.lo ? i : c.rows - (c.keep - i);
    kept[i] = r;
    if (kw != nullptr) kw[i] = r >= 0 ? w[r] : 0.0f;
  }
  if (all || c.take == 0) return;

  // the digits of the last kept row's key, from the top
  uint32_t prefix = 0;                        // key bits above `shift + bits`
  int32_t left = c.take;                      // places for keys with that prefix
  int shift = 21;
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    for (int i = tid; i < kBins; i += kSelectBlock) hist[i] = 0;
    __syncthreads();
    for (int32_t r = c.lo + tid; r < c.hi; r += kSelectBlock) {
      const uint32_t k = weight_key(w[r]);
      if (pass == 0 || k >> (shift + bits) == prefix) atomicAdd(&hist[k >> shift & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    // bins from the greatest down, two a thread
    const int top = (1 << bits) - 1 - 2 * tid;
    const int32_t n0 = top >= 0 ? (int32_t)hist[top] : 0, n1 = top >= 1 ? (int32_t)hist[top - 1] : 0;
    int32_t total;
    const int32_t end = block_scan(n0 + n1, buf[pass & 1], &total);
    const int32_t at = end - n0 - n1;         // keys in greater bins
    if (at < left && at + n0 >= left) found[0] = top, found[1] = left - at;
    else if (at + n0 < left && end >= left) found[0] = top - 1, found[1] = left - at - n0;
    __syncthreads();
    prefix = pass == 0 ? (uint32_t)found[0] : prefix << bits | (uint32_t)found[0];
    left = found[1];
    shift = pass == 0 ? 10 : 0;
  }
  // keys above `prefix` are kept, and the first `left` equal to it
  int32_t above = 0, equal = 0;               // of the rows before this turn's
  int turn = 0;
  for (int32_t r0 = c.lo; r0 < c.hi; r0 += kSelectBlock, turn ^= 1) {
    const int32_t r = r0 + tid;
    const float v = r < c.hi ? w[r] : 0.0f;
    const uint32_t k = weight_key(v);
    const bool gt = r < c.hi && k > prefix, eq = r < c.hi && k == prefix;
    int32_t total;
    // (both counts of a turn fit 16 bits)
    const int32_t end = block_scan((gt ? 1 : 0) | (eq ? 1 << 16 : 0), buf[turn], &total);
    const int32_t before_gt = above + (end & 0xFFFF) - (gt ? 1 : 0);
    const int32_t before_eq = equal + (end >> 16) - (eq ? 1 : 0);
    if (gt || (eq && before_eq < left)) {
      const int32_t i = c.lo + before_gt + min(before_eq, left);
      kept[i] = r;
      if (kw != nullptr) kw[i] = v;
    }
    above += total & 0xFFFF;
    equal += total >> 16;
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
  // few rows are spread over more waves
  const uint32_t batch = rows_at >= (uint32_t)kBatch * kCompactGrid * kCompactWaves ? kBatch : 8;
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
  select_kernel<<<dim3((uint32_t)p.num_slots), kSelectBlock, 0, stream>>>(p);
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
