// slot_map.hip -- block tables and slot maps of a batch from its request
// lengths (gfx950).
//
// One launch.  Every workgroup scans the whole batch -- two prefix sums over
// the slots, pages asked for and tokens added -- into LDS, and then writes
// its share of the per-slot, per-page and per-token outputs; a page or token
// finds its slot by a binary search of the LDS prefixes.  Repeating the scan
// in each workgroup (8 bytes a slot, from the L2 after the first) costs less
// than a second launch.  No workgroup reads what another one writes: the
// page of a token that falls on a page taken in this call is looked up in
// the free list, not in the page table.
//
// It is latency: two dependent loads, a scan and two more take 5.5 to 6.5 us for
// 1,024 decodes as for the 60,000 tokens of 300 requests; the bytes (0.8 MB there)
// would take 0.2.  Past 1,024 slots every further 1,024 add a turn of the scans:
// 4,096 decodes take 10.6 us a call, 8,191 16.4.
#include "launch_attend.hpp"
#include "layout.hpp"
#include "wave.hpp"

namespace kvc {

namespace {

constexpr int kMapBlock = 1024;
constexpr int kMapWaves = kMapBlock / kLanes;
constexpr int kMapSlots = 8192;              // slots the LDS tables hold

// Sums saturate at kSat: a batch may ask for more than 2^32 pages or tokens
// before it is refused, and every accepted sum stays below kSat.
constexpr uint32_t kSat = 0x7FFFFFFF;
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

// inclusive saturating sum over the 64 lanes (values up to kSat), the steps of
// wave_incl_scan_i32
__device__ __forceinline__ uint32_t wave_sat_scan(uint32_t v) {
  v = sat_add(v, (uint32_t)dpp_shr_or_zero<0x111>((int32_t)v));
  v = sat_add(v, (uint32_t)dpp_shr_or_zero<0x112>((int32_t)v));
  v = sat_add(v, (uint32_t)dpp_shr_or_zero<0x114>((int32_t)v));
  v = sat_add(v, (uint32_t)dpp_shr_or_zero<0x118>((int32_t)v));
  v = sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowBcast15, 0xA, 0xF, false));
  return sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowBcast31, 0xC, 0xF, false));
}

// Inclusive saturating sum over the workgroup's threads; *total: of all of
// them.  buf: kMapWaves words that no thread still reads.
__device__ __forceinline__ uint32_t block_sat_scan(uint32_t v, uint32_t* buf, uint32_t* total) {
  const int lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  v = wave_sat_scan(v);
  if (lane == kLanes - 1) buf[wave] = v;
  __syncthreads();
  // every wave sums the waves' totals in its first lanes
  const uint32_t t = wave_sat_scan(lane < kMapWaves ? buf[lane] : 0u);
  *total = (uint32_t)__builtin_amdgcn_readlane((int)t, kLanes - 1);
  return wave == 0 ? v : sat_add(v, (uint32_t)__builtin_amdgcn_readlane((int)t, wave - 1));
}

// Last index i in [0, n) with start[i] <= x (start[0] = 0 <= x, ascending)
__device__ __forceinline__ int last_at_most(const int32_t* start, int n, int32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct SlotPlan {
  int64_t len, n;        // stored and added tokens (added: 0 unless live)
  int64_t have, need;    // pages held, pages to take
  bool live, ok;         // an active slot; not refused so far
};

// Slot b before the shared limits (free pages, token rows) are looked at
__device__ __forceinline__ SlotPlan slot_plan(const SlotMapParams& p, int b, int32_t* bad) {
  SlotPlan s;
  s.len = p.lens[b];
  s.n = p.new_lens != nullptr ? p.new_lens[b] : p.token_stride;
  s.live = s.len >= 0;
  if (!s.live) s.len = 0;
  if (!s.live || s.n < 0) s.n = 0;
  const int rl = p.ratio - 1;                 // log2 of the ratio
  const int64_t ps = int64_t(1) << p.page_bits;
  s.have = ((s.len >> rl) + ps - 1) >> p.page_bits;
  const int64_t want = (((s.len + s.n) >> rl) + ps - 1) >> p.page_bits;
  s.ok = s.live;
  if (want > p.pt_width || s.len + s.n > 0x7FFFFFFF) {
    s.ok = false;
    *bad |= kStPtRange;
  } else if (p.token_stride > 0 && s.n > p.token_stride) {
    s.ok = false;
    *bad |= kStTokenRange;
  }
  if (!s.ok) s.n = 0;
  s.need = s.ok ? want - s.have : 0;
  return s;
}

__global__ __launch_bounds__(kMapBlock) void slot_map_kernel(SlotMapParams p) {
  __shared__ int32_t tok0[kMapSlots];         // first token row of each slot
  __shared__ int32_t page0[kMapSlots];        // its first place in the free list
  __shared__ uint32_t okbits[kMapSlots / 32];
  __shared__ uint32_t buf[2][kMapWaves];
  __shared__ int32_t top[kMapWaves][2], sums[kMapWaves][3];
  const int S = p.num_slots, tid = threadIdx.x, lane = lane_id();
  const int wave = uniform(tid >> 6);
  const int rl = p.ratio - 1;
  const bool first_block = blockIdx.x == 0;
  int32_t bad = 0;
  uint32_t page_carry = 0, tok_carry = 0;
  // accepted places in the free list and token rows, tokens, compressed rows,
  // refused slots: of this thread
  int32_t pages = 0, tokens = 0, n_sum = 0, row_sum = 0, refused = 0;

  // (a turn's scans leave a barrier between any read of buf and the next turn's
  // write of the same words)
  for (int b0 = 0; b0 < S; b0 += kMapBlock) {
    const int b = b0 + tid;
    SlotPlan s{};
    if (b < S) s = slot_plan(p, b, &bad);
    // (need and n are below 2^31: the table and the length were checked)
    uint32_t total;
    const uint32_t pe = sat_add(block_sat_scan((uint32_t)s.need, buf[0], &total), page_carry);
    page_carry = sat_add(page_carry, total);
    if (s.need > 0 && pe > (uint32_t)p.n_free) {
      s.ok = false;
      s.n = 0;
      bad |= kStNoPage;
    }
    // packed tokens are numbered through the batch; with a stride each slot
    // has its own rows, and only their sum is of interest
    const uint32_t te = sat_add(block_sat_scan((uint32_t)s.n, buf[1], &total), tok_carry);
    tok_carry = sat_add(tok_carry, total);
    if (p.token_stride == 0 && s.n > 0 && te > (uint32_t)p.max_tokens) {
      s.ok = false;
      s.n = 0;
      bad |= kStTokenRange;
    }
    const uint64_t okm = __ballot(s.ok);
    if (b < S) {
      // a refused slot's places are cut to the accepted totals below
      page0[b] = (int32_t)(pe == kSat ? kSat : pe - (uint32_t)s.need);
      tok0[b] = (int32_t)(te == kSat ? kSat : te - (uint32_t)s.n);
      if (lane == 0) {
        okbits[b >> 5] = (uint32_t)okm;
        okbits[(b >> 5) + 1] = (uint32_t)(okm >> 32);
      }
      if (s.ok) {
        if (s.need > 0) pages = (int32_t)pe;
        if (s.n > 0) tokens = (int32_t)te;
        n_sum += (int32_t)s.n;
        row_sum += (int32_t)(((s.len + s.n) >> rl) - (s.len >> rl));
      } else if (s.live) {
        ++refused;
      }
    }
  }
  // the accepted totals: the last accepted ends (ascending over the slots, so
  // maxima), and the sums, by waves
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) {
    pages = max(pages, __shfl_xor(pages, d));
    tokens = max(tokens, __shfl_xor(tokens, d));
  }
  if (first_block) {
    n_sum = wave_incl_scan_i32(n_sum);
    row_sum = wave_incl_scan_i32(row_sum);
    refused = wave_incl_scan_i32(refused);
    if (lane == kLanes - 1) { sums[wave][0] = n_sum; sums[wave][1] = row_sum; sums[wave][2] = refused; }
  }
  if (lane == 0) { top[wave][0] = pages; top[wave][1] = tokens; }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMapWaves; ++w) {
    pages = max(pages, top[w][0]);            // packed token rows and pages in use
    tokens = max(tokens, top[w][1]);
  }
  auto accepted = [&](int b) { return (okbits[b >> 5] >> (b & 31) & 1u) != 0; };
  auto added = [&](int b) -> int32_t {
    if (!accepted(b)) return 0;
    const int32_t n = p.new_lens != nullptr ? p.new_lens[b] : p.token_stride;
    return n > 0 ? n : 0;
  };
  for (int b = tid; b < S; b += kMapBlock) {
    if (page0[b] > pages) page0[b] = pages;
    if (tok0[b] > tokens) tok0[b] = tokens;
  }
  __syncthreads();

  const int64_t at = (int64_t)blockIdx.x * kMapBlock + tid, step = (int64_t)gridDim.x * kMapBlock;
  // ---- per slot
  for (int64_t b = at; b < S; b += step) {
    if (p.offsets != nullptr) {
      p.offsets[b] = p.token_stride > 0 ? (int32_t)b * p.token_stride : tok0[b];
      p.offsets[S + b] = added((int)b);
    }
    if (p.start_pos != nullptr) p.start_pos[b] = accepted((int)b) ? p.lens[b] : -1;
  }
  if (first_block && tid == 0 && p.totals != nullptr) {
    int32_t t[3] = {};
    for (int w = 0; w < kMapWaves; ++w)
      for (int i = 0; i < 3; ++i) t[i] += sums[w][i];
    p.totals[0] = t[0];
    p.totals[1] = t[1];
    p.totals[2] = pages;
    p.totals[3] = t[2];
  }
  // ---- per page taken: the slots' places ascend, so the last slot that
  // starts at or below a page is its owner (slots that take none share the
  // start of the one after them and are passed over)
  for (int64_t e = at; e < pages; e += step) {
    const int b = last_at_most(page0, S, (int32_t)e);
    const int64_t ps = int64_t(1) << p.page_bits;
    const int64_t have = (((int64_t)p.lens[b] >> rl) + ps - 1) >> p.page_bits;
    p.page_table[(int64_t)b * p.pt_stride + have + (e - page0[b])] = p.free_pages[e];
  }
  // ---- per token
  for (int64_t t = at; t < p.max_tokens; t += step) {
    int b = -1;
    int32_t j = 0;
    if (p.token_stride > 0) {
      const uint32_t q = udiv_magic((uint32_t)t, p.stride_div.m, p.stride_div.sh1, p.stride_div.sh2);
      if (q < (uint32_t)S) {
        b = (int)q;
        j = (int32_t)t - b * p.token_stride;
        if (j >= added(b)) b = -1;
      }
    } else if (t < tokens) {
      b = last_at_most(tok0, S, (int32_t)t);
      j = (int32_t)t - tok0[b];
    }
    int32_t loc = 0, pos = 0;
    if (b >= 0) {
      const int32_t len = p.lens[b];
      const int32_t q = len + j;
      pos = p.depth != nullptr ? len + p.depth[t] : q;
      if (((q + 1) & rl) == 0) {              // the token closes a row
        const int32_t c = q >> rl, lp = c >> p.page_bits;
        const int32_t have = (int32_t)((((int64_t)len >> rl) + (int64_t(1) << p.page_bits) - 1) >>
                                       p.page_bits);
        const int32_t page = lp < have ? p.page_table[(int64_t)b * p.pt_stride + lp]
                                       : p.free_pages[page0[b] + (lp - have)];
        if (page >= 0 && page < p.num_pages)
          loc = (page << p.page_bits) | (c & ((1 << p.page_bits) - 1));
        else
          bad |= kStPageRange;
      }
    }
    if (p.out_loc != nullptr) p.out_loc[t] = loc;
    if (p.positions != nullptr) p.positions[t] = pos;
    if (p.token_to_req != nullptr) p.token_to_req[t] = b;
  }
  if (bad != 0 && p.status != nullptr) atomicOr(p.status, bad);
}

}  // namespace

hipError_t launch_slot_map(const SlotMapParams& p, hipStream_t stream) {
  // a token or slot a thread, up to the chip's compute units; the LDS tables
  // leave room for one workgroup of this size per unit
  int64_t units = p.max_tokens > p.num_slots ? p.max_tokens : p.num_slots;
  int64_t blocks = (units + kMapBlock - 1) / kMapBlock;
  if (blocks > 256) blocks = 256;
  hipLaunchKernelGGL(slot_map_kernel, dim3((unsigned)(blocks < 1 ? 1 : blocks)), dim3(kMapBlock), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace kvc
