// attend.hip -- attention over the paged compressed cache (gfx950): drafted
// tokens (a tree, a chain, one token) and packed causal prompts.
//
// A cached row x_r is key and value at once (512 dims, one row for all H query
// heads), so for a query q over its visible rows
//   s_r = scale * q . x_r,   out = sum_r e^(s_r) x_r / (sum_r e^(s_r) + e^sink)
// and one staged tile of rows serves both products.
//
// The queries of a slot are its (token, head) pairs in that order, cut into
// units of QT = 32 QB; a unit's rows are cut into tiles of NT = 128 / QB.  The
// tiles of all units are dealt evenly to the workgroups of attend_kernel (one
// per compute unit, each a run of consecutive tiles, crossing units as it
// comes) by attend_plan_kernel, or for few units by each workgroup itself, and
// attend_join_kernel joins the units that were cut between workgroups.  The
// split follows the lengths on the device, so a captured call adapts to
// refreshed lengths, and it is a function of the lengths alone, so results
// repeat bit for bit.
//
// What bounds it: a tile costs 2 * 2 * QT * NT * 512 flops and NT rows of 528
// (V41), 288 (V41_FP4) or 584 (V4) bytes.  At about 1.5 PFLOP/s (the clock falls
// to 1.6 GHz under the matrix units) and 5.2 TB/s the two take the same time at 75
// queries a unit for V41, 41 for V41_FP4 and 83 for V4: units of 128 are bound by
// the matrix units, units of 64 by them for V41_FP4 and by HBM for the others,
// units of 32 by HBM.  What it reaches, in visible (query, row) pairs * 2048
// flops: 1.08 PFLOP/s on a prompt of 8,192 tokens with 128 heads (V41, 8.1 ms),
// 0.69 on 16 prompts of some 2,000 tokens with 32 heads (V41_FP4, 16 tiles a unit
// on average, 1.5 ms), 0.61 to 0.63 on 64 decodes with 64 heads (V41_FP4, 120 to
// 125 us), 2.6 to 2.7 TB/s and 0.56 to 0.58 PFLOP/s on 128 chains of 4 with 16
// heads (V4, 125 to 129 us), 3.0 TB/s on 64 decodes with 32 heads (V41, 101 us).
#include <type_traits>

#include "launch_attend.hpp"
#include "row_ops.hpp"

namespace kvc {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kAttendBlock = 256;            // 4 waves, one per SIMD: 512 registers each
constexpr int kAttendGrid = kAttendWorkgroups;
constexpr int kPlanBlock = 1024;
constexpr int kPlanSlots = 8192;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;

// tokens of slot b and the position of its first one; n = 0 for a slot that
// has none or is skipped
struct SlotTokens {
  int32_t first, n, pos;
};
__device__ __forceinline__ SlotTokens slot_tokens(const AttendParams& p, int b, int32_t* bad) {
  SlotTokens s;
  s.pos = p.start_pos[b];
  if (p.offsets == nullptr) {
    s.first = b * p.draft_len;
    s.n = p.draft_len;
  } else {
    s.first = p.offsets[b];
    s.n = p.offsets[p.num_slots + b];
    if (s.n < 0) s.n = 0;
    if (s.pos >= 0 && s.n > 0 && (s.first < 0 || (int64_t)s.first + s.n > p.q_rows)) {
      s.n = 0;
      *bad |= kStTokenRange;
    }
  }
  if (s.pos < 0) s.n = 0;
  // row and tile indices stay in int32
  if (s.n > 0 && (int64_t)s.pos + s.n > 0x7FFFFFFF - 256) {
    s.n = 0;
    *bad |= kStPosRange;
  }
  return s;
}

__device__ __forceinline__ int64_t units_of(const AttendParams& p, int32_t n, int qt) {
  return ((int64_t)n * p.heads + qt - 1) / qt;
}

// rows the queries [m0, m0 + qt) of a slot may see: the last one's limit
__device__ __forceinline__ int32_t unit_rows(const AttendParams& p, const SlotTokens& s, int32_t m0,
                                             int qt) {
  if (p.tree != nullptr) return s.pos + s.n;
  const int32_t last = min(m0 + qt, s.n * p.heads) - 1;
  const int32_t tok = (int32_t)udiv_magic((uint32_t)last, p.head_div.m, p.head_div.sh1, p.head_div.sh2);
  return (s.pos + tok + 1) >> (p.ratio - 1);
}
// a unit with no row still has its output to write: one empty tile
__device__ __forceinline__ int32_t unit_tiles(int32_t rows, int nt) {
  return rows > 0 ? (rows + nt - 1) / nt : 1;
}

// what a unit costs besides its tiles, in tiles
__device__ __forceinline__ int32_t unit_cost(int nt) { return kAttendUnitRows / nt; }

// ------------------------------------------------------------------ plan
// One workgroup: a prefix sum of the slots' units, then each thread walks an
// equal share of the units twice, to sum their tiles and to place the
// boundaries between the workgroups of attend_kernel.  Latency: 6 us for 32
// units, 16 to 18 for 8,192.
__device__ __forceinline__ int64_t plan_excl_scan(int64_t v, int64_t* buf, int64_t* total) {
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) {
    const int64_t o = __shfl_up(x, d);
    if (lane >= d) x += o;
  }
  __syncthreads();
  if (lane == kLanes - 1) buf[wave] = x;
  __syncthreads();
  int64_t t = 0;
  for (int w = 0; w < kPlanBlock / kLanes; ++w) {
    if (w == wave) x += t;
    t += buf[w];
  }
  *total = t;
  return x - v;
}

__global__ __launch_bounds__(kPlanBlock) void attend_plan_kernel(AttendParams p, int qt, int nt) {
  __shared__ int64_t unit0[kPlanSlots];      // first unit of each slot
  __shared__ int64_t buf[kPlanBlock / kLanes];
  __shared__ int32_t nsplit;
  const int S = p.num_slots, tid = threadIdx.x;
  int32_t bad = 0;
  int64_t carry = 0;
  if (tid == 0) nsplit = 0;
  for (int b0 = 0; b0 < S; b0 += kPlanBlock) {
    const int b = b0 + tid;
    int64_t u = 0;
    if (b < S) {
      const SlotTokens s = slot_tokens(p, b, &bad);
      u = units_of(p, s.n, qt);
    }
    int64_t total;
    const int64_t e = plan_excl_scan(u, buf, &total) + carry;
    if (b < S) unit0[b] = e;
    carry += total;
  }
  __syncthreads();
  if (bad != 0 && p.status != nullptr) atomicOr(p.status, bad);
  const int64_t units = carry;
  const int64_t per = (units + kPlanBlock - 1) / kPlanBlock;
  const int64_t ua = min(units, per * tid), ub = min(units, ua + per);
  // last slot starting at or below unit ua (slots without units share the
  // start of the next one)
  int b_first = 0;
  if (ua < ub) {
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (unit0[mid] <= ua) lo = mid;
      else hi = mid - 1;
    }
    b_first = lo;
  }
  auto walk = [&](auto&& f) {
    int b = b_first;
    int32_t none = 0;
    SlotTokens s{};
    if (ua < ub) s = slot_tokens(p, b, &none);
    for (int64_t u = ua; u < ub; ++u) {
      while (b + 1 < S && unit0[b + 1] <= u) {
        ++b;
        if (b + 1 >= S || unit0[b + 1] > u) s = slot_tokens(p, b, &none);
      }
      const int32_t k = (int32_t)(u - unit0[b]);
      f(b, k, (int64_t)unit_tiles(unit_rows(p, s, k * qt, qt), nt));
    }
  };
  // A unit costs its tiles and its begin and end (unit_cost); a boundary
  // that falls into the latter is moved to the unit's first tile.
  int64_t mine = 0, total = 0;
  walk([&](int, int32_t, int64_t t) { mine += t + unit_cost(nt); });
  int64_t c = plan_excl_scan(mine, buf, &total);
  int64_t quota = (total + kAttendGrid - 1) / kAttendGrid;
  const int64_t least = kAttendLeastRows / nt;
  if (quota < least) quota = least;
  // boundary kAttendGrid, and every one past the last unit: the end
  for (int64_t w = tid; w <= kAttendGrid; w += kPlanBlock)
    if (w * quota >= total) p.starts[w] = AttendStart{S, 0, 0, 0};
  walk([&](int b, int32_t k, int64_t t) {
    const int64_t end = c + unit_cost(nt) + t;
    int64_t cut = 0;                          // first boundary inside the tiles
    int32_t parts = 1;
    for (int64_t w = (c + quota - 1) / quota; w * quota < end && w < kAttendGrid; ++w) {
      const int64_t tile = max(w * quota - c - unit_cost(nt), int64_t(0));
      p.starts[w] = AttendStart{b, k, (int32_t)tile, 0};
      if (tile > 0 && ++parts == 2) cut = w;
    }
    if (parts > 1) p.splits[atomicAdd(&nsplit, 1)] = AttendSplit{b, k, (int32_t)(cut - 1), parts};
    c = end;
  });
  __syncthreads();
  if (tid == 0) p.head->nsplit = nsplit;
}

// ------------------------------------------------------------------ staging
// The 16-byte chunks of a staged row are permuted by XOR with a function of
// the row index, so that both products' reads spread over all 64 banks: the
// scores' read one chunk column of 16 consecutive rows at a time, which the
// four bits keep apart; the transposing reads 64 bytes of 4 consecutive rows,
// which the row's low bits, in the chunk index's upper two, keep apart.
__device__ __forceinline__ uint32_t swz(uint32_t row) { return (row & 3u) << 2 | (row >> 2 & 3u); }

typedef const __attribute__((address_space(3))) uint8_t* lds_cptr;
typedef __attribute__((address_space(3))) uint8_t* lds_ptr;

// The lanes' part of an 8-row group that lies in one page: N loads of 16 dims'
// codes a lane (V4: the last one of bf16 rope dims) with the scale bytes of
// their dims, and their expansion into 8 rows of a tile.  Every load's offsets
// are a base of the lane and a constant.
//   V41      load k: rows 2k, 2k + 1, 32 lanes a row, 16 dims a lane
//   V41_FP4  the same (8 bytes a lane: 16-byte loads would put four chunks a
//            lane to one bank group)
//   V4       8 lanes a row; load k < 4: dims 128k + 16 (lane % 8) -- of load 3
//            the upper lanes' are past the codes, and what they put is
//            overwritten by load 4's rope dims, 8 a lane
template <int L> struct GroupShape;
template <> struct GroupShape<kV41> { static constexpr int kLoads = 4; };
template <> struct GroupShape<kV41Fp4> { static constexpr int kLoads = 4; };
template <> struct GroupShape<kV4> { static constexpr int kLoads = 5; };

template <int L>
struct Group {
  static constexpr int N = GroupShape<L>::kLoads;
  typedef typename std::conditional<L == kV41Fp4, u32x2, u32x4>::type Codes;
  Codes codes[N];
  uint32_t scale[N];

  static __device__ __forceinline__ int row(int k, int lane) {
    return L == kV4 ? lane >> 3 : 2 * k + (lane >> 5);
  }
  // the lane's data and scale offsets, and load k's constants on top of them
  static __device__ __forceinline__ uint32_t data_off(int lane) {
    return L == kV41 ? 16 * lane : L == kV41Fp4 ? 8 * lane
                     : (lane >> 3) * LayoutTraits<L>::kData + 16 * (lane & 7);
  }
  static constexpr uint32_t data_step(int k) {
    return L == kV41 ? 1024 * k : L == kV41Fp4 ? 512 * k : k < 4 ? 128 * k : kNope;
  }
  static __device__ __forceinline__ uint32_t scale_off(int lane) {
    return L == kV41 ? lane >> 1 : L == kV41Fp4 ? lane
                     : (lane >> 3) * LayoutTraits<L>::kScale + ((lane & 7) >> 2);
  }
  static constexpr uint32_t scale_step(int k) {
    return L == kV41 ? 32 * k : L == kV41Fp4 ? 64 * k : k < 4 ? 2 * k : 0;
  }
  // load k of the group whose data and scale parts begin there
  __device__ __forceinline__ void load(const uint8_t* data, const uint8_t* sc, uint32_t doff, uint32_t soff, int k) {
    if constexpr (L == kV41Fp4)
      codes[k] = __builtin_amdgcn_raw_buffer_load_b64(raw_rsrc(data), (int)doff, (int)data_step(k), kCpolSc1);
    else
      codes[k] = __builtin_amdgcn_raw_buffer_load_b128(raw_rsrc(data), (int)doff, (int)data_step(k), kCpolSc1);
    if (L == kV4 && k == 4) return;
    scale[k] = __builtin_amdgcn_raw_buffer_load_b8(raw_rsrc(sc), (int)soff, (int)scale_step(k), kCpolSc1);
  }
  // load k of rows in pages of their own: the lane's data and scale bytes
  __device__ __forceinline__ void load_apart(const uint8_t* data, const uint8_t* sc, int k) {
    codes[k] = *(const Codes*)data;
    scale[k] = *sc;
  }
  // part j of load k, 8 dims, to its row in a tile: the place of the lane's
  // first part in the group, whose bits the other parts and loads change.  odd:
  // the group's first row is an odd multiple of 8 (of the tile).
  static __device__ __forceinline__ uint32_t place(int lane, int odd) {
    const uint32_t r = row(0, lane);
    const uint32_t chunk = L == kV4 ? 2 * (lane & 7) : 2 * (lane & 31);
    return r * 1024 + ((chunk ^ swz(r + 8 * odd)) << 4);
  }
  static constexpr int parts(int k) { return L == kV4 && k == 4 ? 1 : 2; }
  __device__ __forceinline__ uint4 expand(int k, int j) const {
    if constexpr (L == kV41Fp4) return dq_fp4x8(codes[k][j], scale[k]);
    else if (L == kV4 && k == 4) return make_uint4(codes[k][0], codes[k][1], codes[k][2], codes[k][3]);
    else return dq_fp8x8(make_uint2(codes[k][2 * j], codes[k][2 * j + 1]), scale[k]);
  }
  static __device__ __forceinline__ void write(lds_ptr rows, uint32_t place, int lane, int k, int j, uint4 v) {
    // rows 2k ..: bits 3 (from bit 1 of the row) and 0 (bit 2)
    uint32_t at = L == kV4 ? (place ^ (16 * j)) + 256 * k : (place ^ (16 * ((k & 1) << 3 ^ k >> 1 ^ j))) + 2048 * k;
    if (L == kV4 && k == 4)                   // chunks 56 .. 63, from place's chunks 0, 2, .. 14
      at = (place ^ (16 * (((2 * (lane & 7)) ^ (8 + (lane & 7)))))) + 768;
    *(__attribute__((address_space(3))) u32x4*)(rows + at) = u32x4{v.x, v.y, v.z, v.w};
  }
  __device__ __forceinline__ void put(lds_ptr rows, uint32_t place, int lane, int k, int j) const {
    write(rows, place, lane, k, j, expand(k, j));
  }
};

// Where the rows of a slot lie.
template <int L>
struct Rows {
  PagedKV<L> kv;
  const int32_t* table;
  int32_t width;                              // (rows end below 2^31: a wider table is not reached)
  int32_t rows;                               // rows any query of the unit sees

  // page-table entry of row r (clamped into the table: always in bounds)
  __device__ __forceinline__ int32_t entry(int32_t r) const {
    const int32_t lp = r >> kv.page_bits;
    return table[lp < width ? lp : width - 1];
  }
  // whether row r, with its entry, is a row of the cache; flags one that should be
  __device__ __forceinline__ bool valid(int32_t r, int32_t page, int32_t* status) const {
    if (r >= rows) return false;
    const bool in = (r >> kv.page_bits) < width;
    if (in && page >= 0 && page < kv.num_pages) return true;
    if (status != nullptr) atomicOr(status, in ? kStPageRange : kStPtRange);
    return false;
  }
  __device__ __forceinline__ const uint8_t* data(int64_t page, int32_t r) const {
    return kv.base + page * kv.page_stride +
           (int64_t)(r & ((1 << kv.page_bits) - 1)) * LayoutTraits<L>::kData;
  }
  __device__ __forceinline__ const uint8_t* scale(int64_t page, int32_t r) const {
    return kv.base + page * kv.page_stride + ((int64_t)LayoutTraits<L>::kData << kv.page_bits) +
           (int64_t)(r & ((1 << kv.page_bits) - 1)) * LayoutTraits<L>::kScale;
  }
};

// ------------------------------------------------------------------ products
// Matrix instructions written out, so that scores live in the vector
// registers their softmax works in and O in accumulator registers: the
// compiler gives every matrix-instruction result of a kernel of this size to
// the accumulator file, which O fills (256 registers for 128 queries), and
// moves O through the vector registers where it allocates it by itself.
// A result feeding the next instruction's C operand needs no wait.  An operand
// that a vector instruction has just written needs two wait states (WAIT: s_nop
// 1): the compiler keeps some of the queries of units of 32 and 64 in
// accumulator registers and copies them over.  The other operands come from LDS
// and from registers that stay, and need none (1 to 2% of the time).  That rests
// on the registers the compiler allocates: the build reads the assembly and
// stops where a wait state is missing.
// scores_done and out_done give the 16 wait states from a last result to a
// vector instruction that reads it.
template <bool WAIT>
__device__ __forceinline__ void score_mfma(f32x16& sc, bf16x8 x, bf16x8 q, bool first) {
  if (WAIT && first)
    asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(sc) : "v"(x), "v"(q));
  else if (WAIT)
    asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+&v"(sc) : "v"(x), "v"(q));
  else if (first)
    asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(sc) : "v"(x), "v"(q));
  else
    asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+&v"(sc) : "v"(x), "v"(q));
}
__device__ __forceinline__ void out_mfma(f32x16& o, bf16x8 x, bf16x8 w) {
  asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(o) : "v"(x), "v"(w));
}
__device__ __forceinline__ void scores_done(f32x16& sc) { asm("s_nop 15" : "+v"(sc)); }
__device__ __forceinline__ void out_done(f32x16& o) { asm("s_nop 15" : "+a"(o)); }

// max of three, the ordinary one or the NaN-free operand (fmaxf would first
// make each operand canonical)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// the products of two bf16 pairs added to v
__device__ __forceinline__ float dot_pair(float v, uint32_t a, uint32_t b) {
  typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2v, a), __builtin_bit_cast(bf16x2v, b), v,
                                         false);
}
// sum of a bf16 pair added to v
__device__ __forceinline__ float add_pair(float v, uint32_t pair) { return dot_pair(v, pair, 0x3F803F80u); }

// ------------------------------------------------------------------ a query
// What a lane knows of its query, and the softmax state of it
struct Query {
  int32_t tok, head;           // of the slot
  bool ok;                     // a query of the slot (else a copy of its last one)
  int32_t lim;                 // rows below are visible ...
  uint64_t bits;               // ... and of the rows from base on those of bits
  float mx, sum, rsum;         // reference maximum (log2), sums of weights and rounded weights
  float sink;                  // log2
};

__device__ __forceinline__ Query query_of(const AttendParams& p, int b, const SlotTokens& s, int32_t m) {
  Query q;
  const int32_t nq = s.n * p.heads;
  q.ok = m < nq;
  const int32_t mm = q.ok ? m : nq - 1;
  q.tok = (int32_t)udiv_magic((uint32_t)mm, p.head_div.m, p.head_div.sh1, p.head_div.sh2);
  q.head = mm - q.tok * p.heads;
  q.bits = 0;
  if (p.tree != nullptr) {
    q.lim = s.pos;
    q.bits = p.tree[(int64_t)b * p.draft_len + q.tok];
    if (s.n < 64) q.bits &= (uint64_t(1) << s.n) - 1;
  } else {
    q.lim = (s.pos + q.tok + 1) >> (p.ratio - 1);
  }
  q.mx = kNegInf;
  q.sum = q.rsum = 0.0f;
  q.sink = p.sink != nullptr ? p.sink[q.head] * kLog2e : kNegInf;
  return q;
}

// Masks the scores of rows r0 + 8 (i / 4) + 4 h + i % 4 of a block; okw: which
// of its 32 rows are rows of the cache.  Returns whether a row that some query
// does not see gave a score that is not finite (it holds a NaN or an infinity).
__device__ __forceinline__ bool mask_scores(f32x16& sc, const Query& q, int32_t r0, int h, int32_t base,
                                            bool tree, uint32_t okw) {
  bool nf = false;
  // (kept from being computed ahead of the loop, for every tile's registers)
  asm volatile("" : "+v"(h));
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int rl = 8 * (i >> 2) + 4 * h + (i & 3);
    const int32_t r = r0 + rl;
    bool see = r < q.lim;
    if (tree) {
      const uint32_t x = (uint32_t)(r - base);
      see |= x < 64u && (q.bits >> (x & 63u) & 1) != 0;
    }
    see &= (okw >> rl & 1) != 0;
    nf |= !see && !(__builtin_fabsf(sc[i]) < __builtin_inff());
    sc[i] = see ? sc[i] : kNegInf;
  }
  return __ballot(nf) != 0;
}

// A query that sees a row holding a NaN or an infinity is NaN, all of it and
// its lse, wherever the row and the query lie.  A NaN gives a NaN weight and
// does so by itself, and so does a score of +inf (inf - inf).  An infinity whose
// score is -inf has the weight 0, and 0 times it makes NaN of its own dims:
// end_piece widens them to the query.  Where that infinity was zeroed, for the
// sake of a query that does not see the row, sees_bad says so.  (What either finds
// goes to the sums by way of sfac, which is 0 otherwise.)
// (A finite row whose score passes fp32 has the weight 0 and nothing else.)
// FP4 rows hold no infinities: a code times its scale is at most 2,688.
template <int L> constexpr bool kInfinities = L != kV41Fp4;
constexpr float kNaN = __builtin_nanf("");

// zeroes every NaN and infinity of a staged tile of ROWS rows and notes the rows
// that held one, a bit each, in bad; all threads (a wave has consecutive rows),
// with a barrier behind it
template <int ROWS>
__device__ __forceinline__ void zero_not_finite(lds_ptr tile, uint32_t* bad) {
  typedef __attribute__((address_space(3))) u32x4* vec;
  typedef typename std::conditional<ROWS == 32, uint8_t,
      typename std::conditional<ROWS == 64, uint16_t, uint32_t>::type>::type
      Bits __attribute__((may_alias));
  const int wave = uniform((int)(threadIdx.x >> 6)), lane = lane_id();
  const lds_ptr rows = tile + wave * (ROWS / 4) * 1024 + 16 * lane;
  constexpr int B = ROWS == 32 ? 8 : 16;      // rows read ahead
  uint32_t found = 0;
#pragma unroll 1
  for (int r0 = 0; r0 < ROWS / 4; r0 += B) {
    u32x4 v[B];
#pragma unroll
    for (int r = 0; r < B; ++r) v[r] = *(vec)(rows + 1024 * (r0 + r));
#pragma unroll
    for (int r = 0; r < B; ++r) {
      bool any = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if ((v[r][k] & 0x7F80u) == 0x7F80u) v[r][k] &= 0xFFFF0000u, any = true;
        if ((v[r][k] & 0x7F800000u) == 0x7F800000u) v[r][k] &= 0xFFFFu, any = true;
      }
      if (__ballot(any) == 0) continue;
      *(vec)(rows + 1024 * (r0 + r)) = v[r];
      found |= 1u << (r0 + r);
    }
  }
  if (lane == 0) ((Bits*)bad)[wave] = (Bits)found;
  __syncthreads();
}

// whether the query sees one of the rows of bad, a bit each of the 32 from r0,
// that lie in its lane (see mask_scores)
__device__ __forceinline__ bool sees_bad(const Query& q, int32_t r0, int h, int32_t base, bool tree,
                                         uint32_t bad) {
  const int32_t below = min(max(q.lim - r0, 0), 32);
  uint32_t seen = (uint32_t)((uint64_t(1) << below) - 1);
  if (tree) {
    const int32_t to = base - r0;             // where bit 0 of bits stands
    seen |= (uint32_t)(to >= 0 ? q.bits << min(to, 63) : q.bits >> min(-to, 63) & (to > -64 ? ~0ull : 0));
  }
  return (seen & bad & (h != 0 ? 0xF0F0F0F0u : 0x0F0F0F0Fu)) != 0;
}

// Out and lse factors of a query from its complete sums (or, with a cut unit,
// the joined ones)
struct Final {
  float f, lse;
};
__device__ __forceinline__ Final finish(float snk, float mx, float sum, float rsum) {
  const float mm = fmaxf(mx, snk);
  const float e = mx == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mx - mm);
  // (an infinite sink outweighs every row: out is 0, lse infinite)
  const float es = snk == kNegInf ? 0.0f : snk == mm ? 1.0f : __builtin_amdgcn_exp2f(snk - mm);
  const float den = rsum * e + es;            // 0: no row and no sink
  return Final{den == 0.0f ? 0.0f : e / den, mm + __builtin_log2f(sum * e + es)};
}

// ------------------------------------------------------------------ attend
// A workgroup's walk over its tiles, from its start to the next workgroup's:
// the piece at hand (tiles [t0, t1) of unit ub of slot b) and the step to the
// next one.
struct Walk {
  int b, ub;
  int32_t t0, t1, tiles, rows;
  int eb, eub, et;             // the end: slot, unit, tile
  int32_t parts;               // (plan_here) workgroups from this one on in the end's unit
  SlotTokens s;

  __device__ __forceinline__ void piece(const AttendParams& p, int qt, int nt) {
    rows = uniform(unit_rows(p, s, ub * qt, qt));
    tiles = unit_tiles(rows, nt);
    t1 = uniform(b == eb && ub == eub ? et : tiles);
    // plan_here: the workgroup with a unit's first tile tells the join how many
    // workgroups share it
    if (p.plan_units > 0 && t0 == 0 && threadIdx.x == 0)
      p.splits[b * p.plan_units + ub] = AttendSplit{b, ub, (int32_t)blockIdx.x, t1 < tiles ? parts : 1};
  }
  __device__ __forceinline__ void take_slot(const AttendParams& p) {
    int32_t none = 0;
    const SlotTokens c = slot_tokens(p, b, &none);
    s = SlotTokens{uniform(c.first), uniform(c.n), uniform(c.pos)};
  }
  __device__ __forceinline__ bool begin(const AttendParams& p, int qt, int nt) {
    if (p.plan_units > 0) {
      if (!plan_here(p, qt, nt)) return false;
    } else {
      const AttendStart st = p.starts[blockIdx.x], en = p.starts[blockIdx.x + 1];
      b = uniform(st.slot), ub = uniform(st.unit), t0 = uniform(st.tile);
      eb = uniform(en.slot), eub = uniform(en.unit), et = uniform(en.tile);
      if (b < p.num_slots) take_slot(p);
    }
    if (b >= p.num_slots || (b == eb && ub == eub && t0 == et)) return false;
    piece(p, qt, nt);
    return true;
  }
  // The plan without a launch of its own, for few units: each wave sums all of
  // them for itself (plan_units places in every slot, those of a share of
  // consecutive ones per lane), and the lanes whose places hold this
  // workgroup's start and end say so.
  __device__ __forceinline__ bool plan_here(const AttendParams& p, int qt, int nt) {
    constexpr int kShare = kAttendPlanUnits / kLanes;
    int lane = lane_id();
    asm volatile("" : "+v"(lane));            // nothing of the plan is kept over the tiles
    const int U = p.plan_units, N = p.num_slots * U, per = (N + kLanes - 1) / kLanes;
    const bool first = blockIdx.x == 0 && threadIdx.x < kLanes;
    SlotTokens c[kShare];
    int32_t cost[kShare], slot[kShare], unit[kShare], bad = 0;
    int64_t mine = 0;
    slot[0] = (int32_t)udiv_magic((uint32_t)(lane * per), p.plan_div.m, p.plan_div.sh1, p.plan_div.sh2);
    unit[0] = lane * per - slot[0] * U;
#pragma unroll
    for (int j = 0; j < kShare; ++j) {
      if (j > 0) {
        const bool wrap = unit[j - 1] + 1 == U;
        slot[j] = slot[j - 1] + (wrap ? 1 : 0);
        unit[j] = wrap ? 0 : unit[j - 1] + 1;
      }
      const bool in = j < per && slot[j] < p.num_slots;
      c[j] = slot_tokens(p, min(slot[j], p.num_slots - 1), &bad);
      const bool has = in && unit[j] < units_of(p, c[j].n, qt);
      cost[j] = has ? unit_tiles(unit_rows(p, c[j], unit[j] * qt, qt), nt) + unit_cost(nt) : 0;
      mine += cost[j];
      if (first && in && !has) p.splits[slot[j] * U + unit[j]] = AttendSplit{slot[j], unit[j], 0, 0};
    }
    if (bad != 0 && first && p.status != nullptr) atomicOr(p.status, bad);
    int64_t x = mine;
    for (int d = 1; d * per < N; d <<= 1) {
      const int64_t y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    auto lane64 = [](int64_t v, int l) {
      return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int32_t)(v >> 32), l) << 32 |
                       (uint32_t)__builtin_amdgcn_readlane((int32_t)v, l));
    };
    const int64_t total = lane64(x, (N - 1) / per);
    const int64_t quota = max((total + kAttendGrid - 1) / kAttendGrid, (int64_t)(kAttendLeastRows / nt));
    const int64_t goal0 = blockIdx.x * quota, goal1 = goal0 + quota;
    if (goal0 >= total) return false;
    bool h0 = false, h1 = false;
    int32_t b0 = 0, u0 = 0, x0 = 0, b1 = 0, u1 = 0, x1 = 0;
    int64_t k = x - mine, last = 0;
    SlotTokens c0{};
#pragma unroll
    for (int j = 0; j < kShare; ++j) {
      const int64_t end = k + cost[j];
      if (goal0 >= k && goal0 < end) {
        h0 = true, b0 = slot[j], u0 = unit[j], c0 = c[j];
        x0 = (int32_t)max(goal0 - k - unit_cost(nt), (int64_t)0);
      }
      if (goal1 >= k && goal1 < end) {
        h1 = true, b1 = slot[j], u1 = unit[j], last = end - 1;
        x1 = (int32_t)max(goal1 - k - unit_cost(nt), (int64_t)0);
      }
      k = end;
    }
    const int l0 = __builtin_ctzll(__ballot(h0));
    b = __builtin_amdgcn_readlane(b0, l0), ub = __builtin_amdgcn_readlane(u0, l0);
    t0 = __builtin_amdgcn_readlane(x0, l0);
    s.first = __builtin_amdgcn_readlane(c0.first, l0), s.n = __builtin_amdgcn_readlane(c0.n, l0);
    s.pos = __builtin_amdgcn_readlane(c0.pos, l0);
    const uint64_t m1 = __ballot(h1);
    const int l1 = m1 != 0 ? __builtin_ctzll(m1) : 0;
    eb = uniform(m1 != 0 ? __builtin_amdgcn_readlane(b1, l1) : p.num_slots);
    eub = uniform(m1 != 0 ? __builtin_amdgcn_readlane(u1, l1) : 0);
    et = uniform(m1 != 0 ? __builtin_amdgcn_readlane(x1, l1) : 0);
    // (its last tile lies with workgroup last / quota)
    const uint64_t z = lane64(last, l1);
    parts = uniform(1 - (int32_t)blockIdx.x +
                    (int32_t)(z >> 32 == 0 ? (uint32_t)z / (uint32_t)quota : z / (uint64_t)quota));
    return true;
  }
  __device__ __forceinline__ bool next(const AttendParams& p, int qt, int nt) {
    if (b == eb && ub == eub) return false;
    t0 = 0;
    ++ub;
    if ((int64_t)ub * qt >= (int64_t)s.n * p.heads) {
      ub = 0;
      int32_t none = 0;
      // the next slot that has tokens, 64 at a time
      for (int bn = b + 1;; bn += kLanes) {
        if (bn >= p.num_slots) return false;
        SlotTokens c{};
        if (bn + lane_id() < p.num_slots) c = slot_tokens(p, bn + lane_id(), &none);
        const uint64_t has = __ballot(c.n > 0);
        if (has != 0) {
          b = bn + __builtin_ctzll(has);
          break;
        }
      }
      take_slot(p);
    }
    if (b == eb && ub == eub && et == 0) return false;
    piece(p, qt, nt);
    return true;
  }
};

// a barrier that orders LDS only: global stores before it are not waited for
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// sixteen accumulators out of the matrix registers here and not before: all of
// them at once would not fit
__device__ __forceinline__ f32x16 taken(f32x16 v) {
  asm volatile("" : "+a"(v));
  return v;
}

// The end of a piece: the sums of each query over the lanes and waves that
// hold rows of it, then its outputs, or its partial sums for the join.  A lane
// holds four dims of a query at a time: outputs are turned through LDS (area:
// the tiles, 96 KB or more, three blocks of 32 queries) so that a wave writes whole rows; partial
// sums are stored as they lie in the registers, a wave's
// 1 KB at a time, in the order [query block][dim block][quad][wave][lane].
// INF: a NaN among a query's dims makes NaN of them all (see kInfinities).
template <int QB, bool INF>
__device__ __forceinline__ void end_piece(const AttendParams& p, const Walk& w, Query& q,
                                          const f32x16 (&o)[4][QB], int qb, int nb,
                                          float (*ssum)[32 * QB], float (*srsum)[32 * QB],
                                          float* sfac, lds_ptr area) {
  constexpr int NB = 4 / QB, QT = 32 * QB;
  int lane = lane_id();
  asm volatile("" : "+v"(lane));              // nothing of the end is worked out before the tiles
  const int wave = uniform((int)(threadIdx.x >> 6));
  const int ql = lane & 31, h = lane >> 5, qi = qb * 32 + ql;
  q.sum = sum_halves(q.sum);
  q.rsum = sum_halves(q.rsum);
  if (h == 0) { ssum[nb][qi] = q.sum; srsum[nb][qi] = q.rsum; }
  const bool whole = w.t0 == 0 && w.t1 == w.tiles;
  __syncthreads();
  // a part that began inside its unit lies in the workgroup's first place
  const int64_t part = ((int64_t)blockIdx.x * 2 + (w.t0 > 0 ? 0 : 1)) * QT;
  if (!whole) {
    float* const pp = p.part_o + part * kDim + 256 * wave + 4 * lane;
#pragma unroll
    for (int x = 0; x < QB; ++x) {
      bool nan = false;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const f32x16 v = taken(o[d][x]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 y = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
          *(f32x4*)(pp + ((x * 4 + d) * 4 + j) * 1024) = y;
          if constexpr (INF) nan |= __builtin_isunordered(y[0], y[1]) || __builtin_isunordered(y[2], y[3]);
        }
      }
      if (INF && __builtin_expect(nan, false)) sfac[x * 32 + ql] = kNaN;
    }
    if constexpr (INF) lds_barrier();         // (the sums above are still being stored)
  }
  if (nb == 0 && h == 0) {
    float sum = ssum[0][qi], rsum = srsum[0][qi];
#pragma unroll
    for (int x = 1; x < NB; ++x) { sum += ssum[x][qi]; rsum += srsum[x][qi]; }
    if constexpr (INF) sum += sfac[qi], rsum += sfac[qi];
    if (whole) {
      const int32_t m = w.ub * QT + qi;
      float snk = q.sink;
      if constexpr (QB == 4) {                // a register that the wide kernel's tiles need
        const int32_t mc = min(m, w.s.n * p.heads - 1);
        snk = p.sink != nullptr
                  ? p.sink[mc - (int32_t)udiv_magic((uint32_t)mc, p.head_div.m, p.head_div.sh1,
                                                    p.head_div.sh2) * p.heads] * kLog2e
                  : kNegInf;
      }
      const Final f = finish(snk, q.mx, sum, rsum);
      sfac[qi] = f.f;
      if (p.lse != nullptr && m < w.s.n * p.heads) p.lse[(int64_t)w.s.first * p.heads + m] = f.lse;
    } else {
      p.part_ml[part + qi] = make_float4(q.mx, sum, rsum, 0.0f);
    }
  }
  if (!whole) return;
  __syncthreads();
  const int32_t nq = w.s.n * p.heads;
  constexpr int R = QB < 3 ? QB : 3;          // blocks of 32 queries that the area holds
#pragma unroll
  for (int x0 = 0; x0 < QB; x0 += R) {
    if (x0 > 0) __syncthreads();
#pragma unroll
    for (int x = x0; x < min(x0 + R, QB); ++x) {
      const float f = sfac[x * 32 + ql];
      const lds_ptr row = area + (x - x0) * 32768 + ql * 1024 + 8 * h;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const f32x16 v = taken(o[d][x]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {           // chunk 16 wave + 4 d + j, permuted by the row
          const uint32_t at = ((16 * wave + 4 * d + j) ^ (ql & 15)) << 4;
          *(__attribute__((address_space(3))) u32x2*)(row + at) =
              u32x2{pack_bf16(v[4 * j] * f, v[4 * j + 1] * f),
                    pack_bf16(v[4 * j + 2] * f, v[4 * j + 3] * f)};
        }
      }
    }
    __syncthreads();
    for (int x = x0; x < min(x0 + R, QB); ++x) {
      // the wave's 8 rows: its first one's place, then from head to head
      const int32_t m = w.ub * QT + x * 32 + wave * 8;
      int32_t tok = (int32_t)udiv_magic((uint32_t)m, p.head_div.m, p.head_div.sh1, p.head_div.sh2);
      int32_t head = m - tok * p.heads;
      const int rows = min(8, nq - m);
      uint16_t* op = p.out + (int64_t)(w.s.first + tok) * p.out_stride + (int64_t)head * p.out_hstride;
      // (a dot product with zeros is NaN where a value is not finite)
      float probe = 0.0f;
      auto turned = [&](int i) {
        const int r = wave * 8 + i;
        return *(const __attribute__((address_space(3))) u32x4*)(
            area + (x - x0) * 32768 + r * 1024 + ((lane ^ (r & 15)) << 4));
      };
      auto write = [&](int i, u32x4 v) {
        *(u32x4*)(op + 8 * lane) = v;
        op += p.out_hstride;
        if (++head == p.heads) {
          head = 0;
          op += p.out_stride - p.heads * p.out_hstride;
        }
      };
      for (int i = 0; i < rows; ++i) {
        const u32x4 v = turned(i);
        if constexpr (INF)
#pragma unroll
          for (int k = 0; k < 4; ++k) probe = dot_pair(probe, v[k], 0);
        write(i, v);
      }
      if (INF && __builtin_expect(__ballot(probe != probe) != 0, false)) {
        // once more, row by row
        op = p.out + (int64_t)(w.s.first + tok) * p.out_stride + (int64_t)(m - tok * p.heads) * p.out_hstride;
        head = m - tok * p.heads;
        for (int i = 0; i < rows; ++i) {
          const u32x4 v = turned(i);
          bool nan = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) nan |= (v[k] & 0x7FFFu) > 0x7F80u || (v[k] & 0x7FFF0000u) > 0x7F800000u;
          const bool any = __ballot(nan) != 0;
          write(i, any ? u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u} : v);
          if (any && lane == 0 && p.lse != nullptr) p.lse[(int64_t)w.s.first * p.heads + m + i] = kNaN;
        }
      }
    }
  }
}

// One workgroup, one unit's tiles at a time: scores S^T[row][query] = X Q^T
// with each wave on one 32 x 32 block (a lane owns one query, so the softmax
// statistics are per lane), the weights through LDS as bf16, then
// O^T[dim][query] += X^T P^T with each wave on 128 of the 512 dims.  X^T comes
// out of the same LDS tile by transposing reads.
//
// The weights are rounded to bf16 for the matrix product, the one rounding
// before the output's own; the sum they are divided by is of the rounded
// weights, so the division undoes a common part of it, while lse uses the
// exact weights.
//
// This is the kernel for units of 32 (QB = 1) and 64 queries; a query's rows
// are spread over NB waves, which agree on its reference maximum a tile late:
// a tile's weights are taken against the maximum of the tiles before it (which
// moves only when it is passed by 8 in log2: weights up to 2^8 lose nothing in
// fp32, and O is rescaled rarely), and only where a score passes that by more
// than 16 (always in a piece's first tile) are they taken again, after the waves
// have compared.  Two barriers a tile then (QB = 1: three).  QB = 2 has two tile
// buffers and expands the next tile between the products of this one; the
// 128-row tiles of QB = 1 leave room for one.
//
// A wave is alone on its SIMD (O, the queries' fragments and the rows in flight
// take its 512 registers), so its issue slots are what it runs out of: on 64
// decodes with 64 heads over V41_FP4 rows it issues in 53% of its cycles, in 33%
// vector instructions (the expansion of the rows for the most), and the matrix
// units work in 29%.  Deeper read-ahead of the tiles' fragments
// (8 instead of 6 for the scores, 5 instead of 3 for O) measured slower: 127 and
// 131 against 125.5 us.
//
// RUN: pages of 8 rows or more, so that an 8-row group lies in one page; smaller
// pages look up every row.
template <int L, int QB, bool RUN>
__global__ __launch_bounds__(kAttendBlock) __attribute__((amdgpu_waves_per_eu(1, 1)))
void attend_kernel(AttendParams p) {
  constexpr int NB = 4 / QB;
  constexpr int QT = 32 * QB, NT = 32 * NB, TB = NT * 1024;
  constexpr int BUF = QB == 2 ? 2 : 1;
  constexpr int RW = NT / 4;                  // rows a wave stages per tile
  constexpr int G = RW / 8;                   // in groups of 8
  constexpr int PS = NT + 8;                  // elements per query in the weights' tile
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[BUF * TB];
  __shared__ __attribute__((aligned(16))) uint16_t wts[QT * PS];
  __shared__ float smax[NB][QT], ssum[NB][QT], srsum[NB][QT], sfac[QT];
  __shared__ __attribute__((aligned(16))) uint8_t svalid[BUF][16];
  __shared__ __attribute__((aligned(4))) uint8_t sjump[4], snf[4];
  __shared__ uint32_t sbad[NB];               // rows of a tile that are not finite
  const int lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  const int ql = lane & 31, h = lane >> 5;
  const int qb = wave % QB, nb = wave / QB;
  const int qi = qb * 32 + ql;                // the lane's query in the unit
  const float c2 = p.scale_log2;
  const bool tree = p.tree != nullptr;

  // LDS addresses: row ql of the wave's score block, and the transposing reads
  // of its dim blocks (the permutation touches the low 4 bits of a chunk's
  // index only, so a few bases and constant offsets reach every chunk)
  const lds_ptr tiles3 = (lds_ptr)tiles;
  const int i16 = lane & 15, g1 = (lane >> 4) & 1;
  uint32_t kp[8], vp[2][4];
#pragma unroll
  for (int k = 0; k < 8; ++k) kp[k] = (nb * 32 + ql) * 1024 + (((2 * k + h) ^ swz(ql)) << 4);
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int rr = 8 * h + 4 * e + (i16 >> 2);
      const int chunk = (4 * d + 2 * g1 + ((i16 >> 1) & 1)) ^ swz(rr);
      vp[e][d] = rr * 1024 + 256 * wave + (chunk << 4) + 8 * (i16 & 1);
    }
  const uint32_t place = Group<L>::place(lane, G > 1 ? 0 : wave & 1), doff = Group<L>::data_off(lane),
                 soff = Group<L>::scale_off(lane);
  const int32_t width = (int32_t)min(p.pt_width, (int64_t)0x7FFFFFFF);

  Walk w;
  if (!w.begin(p, QT, NT)) return;
  do {
    const int32_t m0 = w.ub * QT;
    Query q = query_of(p, w.b, w.s, m0 + qi);
    const int32_t lim_first = tree ? w.s.pos : uniform(
        (w.s.pos + (int32_t)udiv_magic((uint32_t)m0, p.head_div.m, p.head_div.sh1, p.head_div.sh2) + 1) >>
        (p.ratio - 1));
    const Rows<L> rw{{p.cache.base, p.cache.page_stride, p.cache.num_pages, p.cache.page_bits},
                     p.page_table + (int64_t)w.b * p.pt_stride, width, w.rows};
    const int32_t row0 = wave * RW;           // of the tile: this wave's first row to stage
    auto first_row = [&](int32_t tl) { return min(tl, w.t1 - 1) * NT + row0; };
    auto entry = [&](int32_t tl) { return rw.entry(first_row(tl) + (lane & (RW - 1))); };
    // group g of a tile whose rows' pages are given; the pages' rows that are
    // none load page 0's, which any cache has; they are masked
    Group<L> gr[G];
    constexpr int NL = Group<L>::N;
    uint32_t okm, okm_next;
    int32_t pages, r0;
    auto locate = [&](int32_t tl, int32_t page) {
      r0 = first_row(tl);
      const bool ok = lane < RW && rw.valid(r0 + lane, page, p.status);
      okm_next = (uint32_t)__ballot(ok);
      pages = ok ? page : 0;
    };
    auto load = [&](int g, int k) {
      if constexpr (RUN) {
        const int32_t pg = __builtin_amdgcn_readlane(pages, 8 * g);
        gr[g].load(rw.data(pg, r0 + 8 * g), rw.scale(pg, r0 + 8 * g), doff, soff, k);
      } else {
        const int row = Group<L>::row(k, lane);
        const int64_t pg = __shfl(pages, 8 * g + row);
        const int32_t r = r0 + 8 * g + row;
        gr[g].load_apart(rw.data(pg, r) + (doff + Group<L>::data_step(k) - row * LayoutTraits<L>::kData),
                         rw.scale(pg, r) + (soff + Group<L>::scale_step(k) - row * LayoutTraits<L>::kScale), k);
      }
    };
    auto load_all = [&]() {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int k = 0; k < NL; ++k) load(g, k);
      okm = okm_next;
    };
    auto put = [&](uint32_t buf, int g, int k, int j) {
      gr[g].put(tiles3 + buf + (row0 + 8 * g) * 1024, G > 1 ? place ^ (32 * (g & 1)) : place, lane, k, j);
    };
    auto put_all = [&](uint32_t buf) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int k = 0; k < NL; ++k)
#pragma unroll
          for (int j = 0; j < Group<L>::parts(k); ++j) put(buf, g, k, j);
    };
    auto note_valid = [&](int buf) {
      if (lane < G) svalid[buf][wave * G + lane] = (uint8_t)(okm >> (8 * lane));
    };
    // the table entries of the first tiles and the first tile's rows are asked
    // for before the queries are waited for
    const int32_t page0 = entry(w.t0), page1 = entry(w.t0 + 1);
    int32_t page = entry(w.t0 + 2);
    locate(w.t0, page0);
    load_all();
    bf16x8 qv[32];
    {
      const uint16_t* qp = p.q + (int64_t)(w.s.first + q.tok) * p.q_stride +
                           (int64_t)q.head * p.q_hstride + 8 * h;
#pragma unroll
      for (int k = 0; k < 32; ++k) qv[k] = __builtin_bit_cast(bf16x8, ld_u4(qp + 16 * k));
    }
    put_all(0);
    note_valid(0);
    locate(w.t0 + 1, page1);
    load_all();
    f32x16 o[4][QB];
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int x = 0; x < QB; ++x) o[d][x] = f32x16{};
    if (kInfinities<L> && threadIdx.x < QT) sfac[threadIdx.x] = 0.0f;
    float ref[QB];                            // reference maxima of all the unit's queries ql, 32 + ql
#pragma unroll
    for (int x = 0; x < QB; ++x) ref[x] = kNegInf;
    __syncthreads();

    typedef const __attribute__((address_space(3))) u32x4* vec;
    typedef __attribute__((address_space(3))) s16x4* trp;
    for (int32_t tl = w.t0; tl < w.t1; ++tl) {
      const int par = BUF == 2 ? (tl - w.t0) & 1 : 0;
      const uint32_t cur = par * TB;
      if constexpr (BUF == 1) {
        if (tl > w.t0) {
          // ---- stage the tile's rows, request the next tile's
          put_all(0);
          note_valid(0);
          locate(tl + 1, page);
          page = entry(tl + 2);
          load_all();
          __syncthreads();
        }
      }
      // With two buffers, tile tl + 1 is expanded into the other one in steps
      // between the products (conversions, their write a step later, and the
      // load for tile tl + 2 in the registers that are free then): the first
      // half between the score products, the rest between O's.
      constexpr int PARTS = L == kV4 ? 9 : 2 * NL;      // of a group
      constexpr int HALF = (G * PARTS + 1) / 2;
      uint4 put_v = make_uint4(0, 0, 0, 0);
      auto stage = [&](int part, int step) {  // part: over all groups
        const int g = part / PARTS, r = part % PARTS, k = r >> 1, j = r & 1;
        if (g >= G) return;
        if (step == 0) put_v = gr[g].expand(k, j);
        else if (step == 1)
          Group<L>::write(tiles3 + (cur ^ TB) + (row0 + 8 * g) * 1024,
                          G > 1 ? place ^ (32 * (g & 1)) : place, lane, k, j, put_v);
        else if (j == Group<L>::parts(k) - 1) load(g, k);
      };
      // ---- scores of this wave's 32 rows and 32 queries
      f32x16 sc;
      {
        constexpr int LA = 6;
        bf16x8 x[LA];
        auto rows16 = [&](int k) {
          return __builtin_bit_cast(bf16x8, *(vec)(tiles3 + cur + kp[k & 7] + 32 * (k & ~7)));
        };
#pragma unroll
        for (int k = 0; k < LA; ++k) x[k] = rows16(k);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          score_mfma<true>(sc, x[k % LA], qv[k], k == 0);
          if (k + LA < 32) x[k % LA] = rows16(k + LA);
          if constexpr (BUF == 2) {
            if (k == 1) note_valid(par ^ 1);
            if (k == 2) locate(tl + 2, page);
            if (k == 4) page = entry(tl + 3);
            if (k >= 5 && (k - 5) / 3 < HALF) stage((k - 5) / 3, (k - 5) % 3);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      scores_done(sc);
      // ---- mask (only a tile that some query does not see whole)
      bool holes = (tl + 1) * NT > lim_first;
#pragma unroll
      for (int x = 0; x < NB; ++x) holes |= uniform(*(const int32_t*)(svalid[par] + 4 * x)) != -1;
      if (holes) {
        const bool any = mask_scores(sc, q, tl * NT + nb * 32, h, w.s.pos, tree,
                                     *(const uint32_t*)(svalid[par] + 4 * nb));
        if (lane == 0) snf[wave] = any;
      }
      // ---- the block's maximum
      float tm = max3(max3(max3(sc[0], sc[1], sc[2]), sc[3], sc[4]),
                      max3(max3(sc[5], sc[6], sc[7]), sc[8], sc[9]),
                      max3(max3(sc[10], sc[11], sc[12]), max3(sc[13], sc[14], sc[15]), sc[15]));
      tm = max_halves(tm) * c2;
      smax[nb][qi] = tm;                      // (both halves of the wave write the same)
      const float mine = QB == 1 || qb == 0 ? ref[0] : ref[QB - 1];
      const bool jump = __ballot(tm > mine + 16.0f) != 0;
      if (lane == 0) sjump[wave] = jump;
      // ---- weights, their sums, and their bf16 to LDS
      uint16_t* const wrow = wts + qi * PS + nb * 32 + 4 * h;
      float ts, tr;
      auto weigh = [&](float at) {
        const float base = at == kNegInf ? 0.0f : at;
        float e[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = __builtin_fmaf(sc[i], c2, -base);
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = __builtin_amdgcn_exp2f(e[i]);
        float t[4] = {};
        tr = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] += e[4 * j + i];
          const uint32_t w0 = pack_bf16(e[4 * j], e[4 * j + 1]), w1 = pack_bf16(e[4 * j + 2], e[4 * j + 3]);
          *(u32x2*)(wrow + 8 * j) = u32x2{w0, w1};
          tr = add_pair(add_pair(tr, w0), w1);
        }
        ts = (t[0] + t[1]) + (t[2] + t[3]);
      };
      weigh(mine);
      __syncthreads();
      // ---- the tile's maxima over the waves of each query, and what the waves noted
      union Frag { s16x4 half[2]; bf16x8 v; };
      auto dims = [&](int i) {                // dim block i & 3, rows 16 (i >> 2) ..
        Frag f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          f.half[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (trp)(tiles3 + cur + vp[e][i & 3] + 16384 * (i >> 2)));
        return f.v;
      };
      auto weights = [&](int k, int x) {
        return __builtin_bit_cast(bf16x8, *(const u32x4*)(wts + (x * 32 + ql) * PS + 16 * k + 8 * h));
      };
      const int32_t jumps = *(const int32_t*)sjump, bad = *(const int32_t*)snf;
      float top[QB], part[QB][NB];
#pragma unroll
      for (int x = 0; x < QB; ++x)
#pragma unroll
        for (int y = 0; y < NB; ++y) part[x][y] = smax[y][x * 32 + ql];
      constexpr int N = NT / 4;               // dim blocks times 16-row steps
      bf16x8 xv[3], wv[2][QB];
      auto first_frags = [&]() {
#pragma unroll
        for (int x = 0; x < QB; ++x) wv[0][x] = weights(0, x);
#pragma unroll
        for (int i = 0; i < 3; ++i) xv[i] = dims(i);
      };
      first_frags();
#pragma unroll
      for (int x = 0; x < QB; ++x) {
        top[x] = part[x][0];
#pragma unroll
        for (int y = 1; y < NB; ++y) top[x] = fmaxf(top[x], part[x][y]);
      }
      const bool again = uniform(jumps) != 0, dirty = holes && uniform(bad) != 0;
      // raises the references passed by more than 8 and rescales what was summed
      auto raise = [&]() {
#pragma unroll
        for (int x = 0; x < QB; ++x) {
          if (tl == w.t0) {                   // (nothing is summed yet)
            ref[x] = top[x];
            continue;
          }
          if (__ballot(top[x] > ref[x] + 8.0f) == 0) continue;
          const float old = ref[x];
          if (top[x] > old + 8.0f) ref[x] = top[x];
          const float alpha = ref[x] == old ? 1.0f : __builtin_amdgcn_exp2f(old - ref[x]);
          if (x == qb) {
            q.sum *= alpha;
            q.rsum *= alpha;
          }
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            out_done(o[d][x]);
            o[d][x] *= alpha;
          }
        }
      };
      if (again || dirty) {
        if (again) {
          raise();
          weigh(QB == 1 || qb == 0 ? ref[0] : ref[QB - 1]);
        }
        // a NaN or an infinity in a row that some query does not see: its weight
        // there is 0, and 0 times it would not be
        if (__builtin_expect(dirty, false)) {
          zero_not_finite<NT>(tiles3 + cur, sbad);
          if (kInfinities<L> && sees_bad(q, tl * NT + nb * 32, h, w.s.pos, tree,
                                         sbad[nb] & *(const uint32_t*)(svalid[par] + 4 * nb)))
            sfac[qi] = kNaN;
        }
        __syncthreads();
        first_frags();
      }
      q.sum += ts;
      q.rsum += tr;
      // ---- O += X^T P^T on dims [128 wave, 128 wave + 128)
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int x = 0; x < QB; ++x) {
          out_mfma(o[i & 3][x], xv[i % 3], wv[(i >> 2) & 1][x]);
          if (x == QB - 1 && i + 3 < N) xv[i % 3] = dims(i + 3);
          if ((i & 3) == 1 && i + 4 < N) wv[((i >> 2) + 1) & 1][x] = weights((i >> 2) + 1, x);
          if constexpr (BUF == 2) {
            const int step = i * QB + x;
            stage(HALF + step / 3, step % 3);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if constexpr (BUF == 2) okm = okm_next;
      if (!again) raise();
      __syncthreads();                        // the tile, the weights and the maxima are free
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int x = 0; x < QB; ++x) out_done(o[d][x]);
    q.mx = QB == 1 || qb == 0 ? ref[0] : ref[QB - 1];
    end_piece<QB, kInfinities<L>>(p, w, q, o, qb, nb, ssum, srsum, sfac, tiles3);
    __syncthreads();
  } while (w.next(p, QT, NT));
}

// The kernel for 128 queries a unit (QB = 4): the same products, arranged so
// that the matrix instructions follow one another.  A wave is alone on its
// SIMD and issues in order, so everything else is placed by hand between
// them: the next tile's expansion and the loads after it between the score
// products, the softmax of this tile between the O products of the previous
// one.  That takes three tile buffers and two of weights, and one barrier a
// tile.  Pages of 8 rows or more.
//
// On a prompt of 8,192 tokens with 128 heads (V41) the matrix units work in
// half of the cycles (64 products of 32 cycles in a tile's 4,000 or so), at 1.08
// PFLOP/s.  The registers are full: a value more that lives over the tiles, or
// accumulators that leave the matrix registers all at once, spills inside the
// loop and cost 10% (9.2 against 8.2 ms).
template <int L>
__global__ __launch_bounds__(kAttendBlock) __attribute__((amdgpu_waves_per_eu(1, 1)))
void attend_wide_kernel(AttendParams p) {
  constexpr int QB = 4, QT = 128, NT = 32, PS = NT + 8, TB = NT * 1024, WB = QT * PS * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[3 * TB];
  __shared__ __attribute__((aligned(16))) uint8_t wts[2 * WB];
  constexpr int kTail = 8;
  __shared__ __attribute__((aligned(16))) uint8_t qtail[4 * kTail * 1024];
  __shared__ float ssum[1][QT], srsum[1][QT], sfac[QT], salpha[2][QT];
  // a byte a wave: the tile's valid 8-row groups, the rescaled query blocks, the
  // blocks that met a score that is not finite where it is masked
  __shared__ __attribute__((aligned(4))) uint8_t svalid[2][4], sscale[2][4], snf[2][4];
  // rows of a tile that are not finite, valid rows of a masked tile
  __shared__ uint32_t sbad[1], smasked[2];
  const int lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  const int ql = lane & 31, h = lane >> 5;
  const int qi = wave * 32 + ql;
  const float c2 = p.scale_log2;
  const bool tree = p.tree != nullptr;
  const lds_ptr tiles3 = (lds_ptr)tiles, wts3 = (lds_ptr)wts;
  const int i16 = lane & 15, g1 = (lane >> 4) & 1;
  // LDS offsets within a tile (see attend_kernel); other chunks by XOR
  const uint32_t kbase = ql * 1024 + ((h ^ swz(ql)) << 4);
  uint32_t vbase[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int rr = 8 * h + 4 * e + (i16 >> 2);
    vbase[e] = rr * 1024 + 256 * wave + (((2 * g1 + ((i16 >> 1) & 1)) ^ swz(rr)) << 4) + 8 * (i16 & 1);
  }
  const uint32_t place = Group<L>::place(lane, wave & 1), doff = Group<L>::data_off(lane),
                 soff = Group<L>::scale_off(lane);

  const int32_t width = (int32_t)min(p.pt_width, (int64_t)0x7FFFFFFF);

  Walk w;
  if (!w.begin(p, QT, NT)) return;
  do {
    const int32_t m0 = w.ub * QT;
    Query q = query_of(p, w.b, w.s, m0 + qi);
    const int32_t lim_first = tree ? w.s.pos : uniform(
        (w.s.pos + (int32_t)udiv_magic((uint32_t)m0, p.head_div.m, p.head_div.sh1, p.head_div.sh2) + 1) >>
        (p.ratio - 1));
    const Rows<L> rw{{p.cache.base, p.cache.page_stride, p.cache.num_pages, p.cache.page_bits},
                     p.page_table + (int64_t)w.b * p.pt_stride, width, w.rows};
    // the wave's 8-row group of tile tl lies in one page
    auto first_row = [&](int32_t tl) { return min(tl, w.t1 - 1) * NT + wave * 8; };
    auto entry = [&](int32_t tl) { return rw.entry(first_row(tl)); };
    const uint8_t *ldata, *lscale;            // of the tile being loaded
    auto locate = [&](int32_t tl, int32_t page) -> bool {
      const int32_t r0 = first_row(tl);
      // a group of a page that is none loads page 0's rows; they are masked
      // (one lane asks, so that a bad page is flagged once)
      page = uniform(page);
      const bool in = (r0 >> p.cache.page_bits) < width, ok = in && page >= 0 && page < p.cache.num_pages;
      if (!ok && r0 < w.rows) raise_status(p.status, in ? kStPageRange : kStPtRange);
      ldata = rw.data(ok ? page : 0, r0);
      lscale = rw.scale(ok ? page : 0, r0);
      return ok;
    };
    Group<L> gr;
    constexpr int NL = Group<L>::N;
    // the table entries of the first three tiles, then the first tile's rows,
    // are asked for before the queries are waited for
    const int32_t page0 = entry(w.t0), page1 = entry(w.t0 + 1);
    int32_t page = entry(w.t0 + 2);
    bool valid = locate(w.t0, page0);         // of the tile in gr
#pragma unroll
    for (int k = 0; k < NL; ++k) gr.load(ldata, lscale, doff, soff, k);
    // the queries' fragments: the last kTail of them in LDS (the registers do not
    // hold all beside the rest)
    bf16x8 qv[32 - kTail];
    {
      const uint16_t* qp = p.q + (int64_t)(w.s.first + q.tok) * p.q_stride +
                           (int64_t)q.head * p.q_hstride + 8 * h;
#pragma unroll
      for (int k = 0; k < 32 - kTail; ++k) qv[k] = __builtin_bit_cast(bf16x8, ld_u4(qp + 16 * k));
#pragma unroll
      for (int k = 0; k < kTail; ++k)
        *(u32x4*)(qtail + (wave * kTail + k) * 1024 + 16 * lane) = *(const u32x4*)(qp + 16 * (32 - kTail + k));
    }
#pragma unroll
    for (int k = 0; k < NL; ++k)
#pragma unroll
      for (int j = 0; j < Group<L>::parts(k); ++j) gr.put(tiles3 + wave * 8192, place, lane, k, j);
    if (lane == 0) svalid[0][wave] = valid ? 0xFF : 0;
    valid = locate(w.t0 + 1, page1);
#pragma unroll
    for (int k = 0; k < NL; ++k) gr.load(ldata, lscale, doff, soff, k);
    f32x16 o[4][QB];
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int x = 0; x < QB; ++x) o[d][x] = f32x16{};
    if (kInfinities<L> && threadIdx.x < QT) sfac[threadIdx.x] = 0.0f;
    __syncthreads();

    typedef const __attribute__((address_space(3))) u32x4* vec;
    typedef __attribute__((address_space(3))) s16x4* trp;
    f32x16 sc;
    bf16x8 x[6];                              // row fragments ahead of the score products
    bf16x8 wv[QB], xv[2];                     // weights, dim fragments ahead of the O products
    uint32_t kp[8];                           // the tile's chunk columns
    bool holes = false, holes_before = false;
    uint32_t okg, cuts, okw = 0, cutw = 0;    // svalid, sscale as words, and uniform
    // (lane bases opaque to the compiler, which would otherwise keep what is
    // derived from them in registers of its own)
    auto fresh = [](uint32_t v) { asm volatile("" : "+v"(v)); return v; };
    auto score_rows = [&](int k) {
      return __builtin_bit_cast(bf16x8, *(vec)(tiles3 + kp[k & 7] + 32 * (k & ~7)));
    };
    auto query_tail = [&](int k) {
      return __builtin_bit_cast(bf16x8, *(vec)((lds_cptr)qtail + (wave * kTail + k - (32 - kTail)) * 1024 + 16 * fresh(lane)));
    };
    // the first fragments of the tile at cur, and what was noted of it and of
    // the tile before (parity par: the tile's)
    auto ahead = [&](int i, uint32_t cur, int32_t par) {
      if (i == 0) {
        const uint32_t kb = fresh(kbase);
#pragma unroll
        for (int k = 0; k < 8; ++k) kp[k] = (kb ^ (32 * k)) + cur;
        okg = *(const uint32_t*)svalid[par];
        cuts = *(const uint32_t*)sscale[par ^ 1];
      }
      x[i] = score_rows(i);
    };
    union Frag { s16x4 half[2]; bf16x8 v; };
    uint32_t vb[2], wread;
    auto out_dims = [&](int i, uint32_t at) { // dim block i & 3, rows 16 (i >> 2) ..
      Frag f;
#pragma unroll
      for (int y = 0; y < 2; ++y)
        f.half[y] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (trp)(tiles3 + (vb[y] ^ (64 * (i & 3))) + at + 16384 * (i >> 2)));
      return f.v;
    };
    auto out_weights = [&](int i, int y, int32_t par) {
      return __builtin_bit_cast(bf16x8, *(vec)(wts3 + par * WB + wread + y * 64 * PS + 32 * i));
    };
    // the first fragments of O's products: the tile at `at`, weights of parity par
    auto out_ahead = [&](int i, uint32_t at, int32_t par) {
      if (i == 0) {
        vb[0] = fresh(vbase[0]), vb[1] = fresh(vbase[1]);
        const uint32_t ln = fresh(lane);
        wread = (ln & 31) * (2 * PS) + 16 * (ln >> 5);
        xv[0] = out_dims(0, at);
      } else if (i == 1) {
        wv[0] = out_weights(0, 0, par), wv[1] = out_weights(0, 1, par);
      } else if (i == 2) {
        wv[2] = out_weights(0, 2, par), wv[3] = out_weights(0, 3, par);
      } else {
        xv[1] = out_dims(1, at);
      }
    };
    // Finding tile tl + 2's rows (whose table entry is in page) and asking for
    // tile tl + 3's entry, in steps between the score products.  ldata, lscale:
    // where the rows lie; valid_next: whether they are rows of the cache.
    bool valid_next = false, in_table = false;
    int64_t page_off = 0;
    int32_t next_row = 0;
    auto locate_step = [&](int k, int32_t tl) {
      if (k == 2) {
        next_row = first_row(tl + 2);
        page = uniform(page);
        in_table = (next_row >> p.cache.page_bits) < width;
      } else if (k == 3) {
        valid_next = in_table && page >= 0 && page < p.cache.num_pages;
        if (!valid_next && next_row < w.rows) raise_status(p.status, in_table ? kStPageRange : kStPtRange);
      } else if (k == 5) {
        page_off = (int64_t)(valid_next ? page : 0) * p.cache.page_stride;
      } else if (k == 7) {
        next_row &= (1 << p.cache.page_bits) - 1;
        ldata = p.cache.base + page_off;
      } else if (k == 9) {
        lscale = ldata + ((int64_t)LayoutTraits<L>::kData << p.cache.page_bits);
      } else if (k == 11) {
        ldata += (int64_t)next_row * LayoutTraits<L>::kData;
      } else if (k == 13) {
        lscale += (int64_t)next_row * LayoutTraits<L>::kScale;
      } else if (k == 15) {
        page = entry(tl + 3);
      } else if (k == 18) {
        if (lane == 0) svalid[((tl - w.t0) & 1) ^ 1][wave] = valid ? 0xFF : 0;
        valid = valid_next;
      } else if (k == 20) {
        // what was noted of this tile and of the one before
        okw = (uint32_t)uniform((int32_t)okg);
        cutw = (uint32_t)uniform((int32_t)cuts);
        holes_before = holes;
        holes = (tl + 1) * NT > lim_first || okw != 0xFFFFFFFFu;
      }
    };
    // ---- scores of tile tl at cur (its first fragments in x); at the end the
    // first fragments of O's products over the tile before are read
    auto scores = [&](int32_t tl, uint32_t before) {
      bf16x8 qt[3];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        score_mfma<false>(sc, x[k % 6], k < 32 - kTail ? qv[k < 32 - kTail ? k : 0] : qt[k % 3], k == 0);
        if (k + 3 >= 32 - kTail && k + 3 < 32) qt[k % 3] = query_tail(k + 3);
        if (k + 6 < 32) x[k % 6] = score_rows(k + 6);
        if (k >= 28) out_ahead(k - 28, before, ((tl - w.t0) & 1) ^ 1);
        locate_step(k, tl);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // ---- mask (only a tile that some query does not see whole)
    auto mask = [&](int32_t tl) {
      if (!holes) return;
      scores_done(sc);
      const bool any = mask_scores(sc, q, tl * NT, h, w.s.pos, tree, okw);
      if (lane == 0) snf[(tl - w.t0) & 1][wave] = any;
      if (kInfinities<L>) smasked[(tl - w.t0) & 1] = okw; // (the same of every wave)
    };
    // ---- tile tl + 1 expanded into the buffer at nxt, in steps of their own for
    // the conversions and the write that waits for them, and each load asked for
    // again (tile tl + 2) when it has been used
    uint32_t pl = 0;
    uint4 put_v = make_uint4(0, 0, 0, 0);
    auto stage = [&](int step, uint32_t nxt) {
      if (step == 0) pl = fresh(place);
      const int part = step / 3, k = part >> 1, j = part & 1;
      if (k >= NL || j >= Group<L>::parts(k)) return;
      if (step % 3 == 0) put_v = gr.expand(k, j);
      if (step % 3 == 1) Group<L>::write(tiles3 + nxt + wave * 8192, pl, lane, k, j, put_v);
      if (step % 3 == 2 && j == Group<L>::parts(k) - 1) gr.load(ldata, lscale, doff, soff, k);
    };
    // ---- the softmax of a tile in 28 steps: the maximum, then a weight a step,
    // each operation a step after the one it waits for
    float tm = 0, ref = 0, alpha = 0, swapped = 0, e[16];
    uint32_t wwrite = 0, pair0 = 0, pair1 = 0;
    auto soften = [&](int step, int32_t par) {
      if (step == 1) scores_done(sc);
      if (step >= 1 && step < 5) {
        const int i = 4 * (step - 1);
        tm = step == 1 ? max3(sc[0], sc[1], sc[2]) : max3(tm, sc[i - 1], sc[i]);
        tm = step == 1 ? tm : max3(tm, sc[i + 1], sc[i + 2]);
      }
      if (step == 5) {
        tm = max3(tm, sc[15], sc[15]);
        const uint32_t ln = fresh(lane);
        wwrite = ((ln & 31) + 32 * wave) * (2 * PS) + 8 * (ln >> 5);
      }
      if (step == 6) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(tm), __float_as_uint(tm), false, false);
        tm = __uint_as_float(r[0]), swapped = __uint_as_float(r[1]);
      }
      if (step == 7) tm = max3(tm, swapped, swapped) * c2;
      if (step == 8) {
        // the reference maximum moves only when it is passed by 8 (in log2): weights
        // up to 2^8 lose nothing in fp32, and O is rescaled rarely
        alpha = q.mx;
        q.mx = tm > q.mx + 8.0f ? tm : q.mx;
      }
      if (step == 9) {
        ref = q.mx == kNegInf ? 0.0f : q.mx;
        tm = __builtin_amdgcn_exp2f(alpha - q.mx);
      }
      if (step == 11) {
        alpha = alpha == q.mx ? 1.0f : tm;
        q.sum *= alpha;
        q.rsum *= alpha;
      }
      if (step == 12) {
        const bool rescale = __ballot(alpha != 1.0f) != 0;
        const uint32_t ln = fresh(lane);
        // (both halves of the wave write the same values)
        salpha[par][wave * 32 + (ln & 31)] = alpha;
        sscale[par][wave] = rescale ? 1 : 0;
      }
      // weight i: its exponent at step 10 + i, its power a step later, its sum
      // another one later; a quad's bf16 and its write behind them
      if (step >= 10 && step < 26) e[step - 10] = __builtin_fmaf(sc[step - 10], c2, -ref);
      if (step >= 11 && step < 27) e[step - 11] = __builtin_amdgcn_exp2f(e[step - 11]);
      if (step >= 12 && step < 28) q.sum += e[step - 12];
      if (step >= 15 && step < 28 && (step & 3) == 3) {
        const int i = step - 15;
        pair0 = pack_bf16(e[i], e[i + 1]), pair1 = pack_bf16(e[i + 2], e[i + 3]);
        *(__attribute__((address_space(3))) u32x2*)(wts3 + par * WB + wwrite + 4 * i) = u32x2{pair0, pair1};
      }
      if (step >= 16 && step <= 28 && (step & 3) == 0) q.rsum = add_pair(add_pair(q.rsum, pair0), pair1);
    };
    // ---- what must precede O's products over tile tl at `at` (parity par)
    auto out_begin = [&](int32_t tl, uint32_t at, int32_t par, bool dirty) {
      // a NaN or an infinity in a row that some query does not see: its weight
      // there is 0, and 0 times it would not be
      if (__builtin_expect(dirty && uniform(*(const int32_t*)snf[par]) != 0, false)) {
        zero_not_finite<NT>(tiles3 + at, sbad);
        if (kInfinities<L> && sees_bad(q, tl * NT, h, w.s.pos, tree, sbad[0] & smasked[par])) sfac[qi] = kNaN;
#pragma unroll
        for (int i = 0; i < 4; ++i) out_ahead(i, at, par);
      }
      if (cutw == 0) return;
#pragma unroll
      for (int y = 0; y < QB; ++y) {
        if ((cutw >> (8 * y) & 0xFF) == 0) continue;
        const float a = salpha[par][y * 32 + ql];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          out_done(o[d][y]);
          o[d][y] *= a;
        }
      }
    };
    // ---- O += X^T P^T of the tile at `at` with the weights of parity par, on dims
    // [128 wave, 128 wave + 128); with = true: between them the softmax of the
    // next tile, the expansion of the one after it (at nxt), the barrier after
    // both and this tile's last reads, and the first fragments at nxt
    auto out = [&](uint32_t at, int32_t par, uint32_t nxt, auto with) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bf16x8 xi = xv[i & 1];
#pragma unroll
        for (int y = 0; y < QB; ++y) {
          out_mfma(o[i & 3][y], xi, wv[y]);
          if (y == 0 && i + 2 < 8) xv[i & 1] = out_dims(i + 2, at);
          if (i == 3) wv[y] = out_weights(1, y, par);
          if constexpr (with.value) {
            soften(4 * i + y, par ^ 1);
            stage(4 * i + y, nxt);
            if (i == 7 && y == 0) __syncthreads();
            if (i == 7 && y > 0) {
              ahead(2 * y - 2, nxt, par);
              ahead(2 * y - 1, nxt, par);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    auto after = [](uint32_t at) { return at == 2 * TB ? 0u : at + TB; };
    uint32_t cur = 0;                         // offset of the tile at hand in tiles
#pragma unroll
    for (int i = 0; i < 6; ++i) ahead(i, cur, 0);
    scores(w.t0, cur);
    mask(w.t0);
#pragma unroll
    for (int i = 0; i < 29; ++i) {
      soften(i, 0);
      stage(i, after(cur));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 6; ++i) ahead(i, after(cur), 1);
    for (int32_t tl = w.t0 + 1; tl < w.t1; ++tl) {
      const int32_t par = (tl - w.t0) & 1;
      const uint32_t before = cur;
      cur = after(cur);
      scores(tl, before);
      mask(tl);
      out_begin(tl - 1, before, par ^ 1, holes_before);
      out(before, par ^ 1, after(cur), std::true_type{});
    }
    cutw = (uint32_t)uniform((int32_t)cuts);
    const int32_t last = (w.t1 - 1 - w.t0) & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) out_ahead(i, cur, last);
    out_begin(w.t1 - 1, cur, last, holes);
    out(cur, last, 0, std::false_type{});
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int y = 0; y < QB; ++y) out_done(o[d][y]);
    end_piece<QB, kInfinities<L>>(p, w, q, o, wave, 0, ssum, srsum, sfac, tiles3);
    __syncthreads();
  } while (w.next(p, QT, NT));
}

// ------------------------------------------------------------------ join
// One workgroup per 8 queries and 256 dims (the dims of two waves) of a unit
// that was cut, 8 threads of neighbouring queries on 128 bytes of a part: the
// parts' weights against the common maximum into LDS, then the weighted sum of
// the parts, four dims of each wave a thread.  Bound by the partial sums, 2 KB a
// query and part, that it reads: some 260 parts of 64 queries, 34 MB, take 10 to
// 12 us; 8 parts of 32 queries 4 us, which is latency.  (128 dims a workgroup: 128
// chains of 4 128.5 instead of 125.2 us in all, one decode 21.3 instead of 21.6;
// 512: 126.7 and 22.0.)
constexpr int kJoinWaves = 2;
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p, int qt) {
  __shared__ float weight[kAttendGrid][8];
  __shared__ float red[3][4][8];
  if (p.plan_units == 0 && (int)blockIdx.x >= p.head->nsplit) return;
  const AttendSplit sp = p.splits[blockIdx.x];
  if (sp.parts < 2) return;
  int32_t none = 0;
  const SlotTokens s = slot_tokens(p, sp.slot, &none);
  const int q8 = threadIdx.x & 7, piece = threadIdx.x >> 3, wave = uniform((int)(threadIdx.x >> 6));
  const int32_t m0 = sp.unit * qt + blockIdx.y * 8;
  if (m0 >= s.n * p.heads) return;
  const int qi = blockIdx.y * 8 + q8;         // of the unit
  // part k lies with workgroup wg0 + k: its second place for the first part
  // (which began at the unit's first tile), its first place for the others
  auto place = [&](int k) -> int64_t { return ((int64_t)(sp.wg0 + k) * 2 + (k == 0 ? 1 : 0)) * qt; };
  // The first parts' sums are asked for at once, and all their statistics.
  // piece = dim block * 8 + quad * 2 + half, as the parts are laid out
  constexpr int P = 4, W = kJoinWaves;
  const int x = qi >> 5, ql = qi & 31, w0 = blockIdx.z * W;
  const float* const src = p.part_o + (x * 16 + (piece >> 1)) * 1024 + 256 * w0 + ((piece & 1) * 32 + ql) * 4;
  float4 ml[kAttendGrid / 32];
#pragma unroll
  for (int i = 0; i < kAttendGrid / 32; ++i) {
    const int k = piece + 32 * i;
    ml[i] = make_float4(kNegInf, 0.0f, 0.0f, 0.0f);
    if (k < sp.parts) ml[i] = p.part_ml[place(k) + qi];
  }
  f32x4 v[P][W];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float* const part = src + place(min(i, sp.parts - 1)) * kDim;
#pragma unroll
    for (int w = 0; w < W; ++w) v[i][w] = *(const f32x4*)(part + 256 * w);
  }
  // over the 8 lanes of a query in each wave, then over the waves
  auto spread = [&](float y, int slot, auto op) {
#pragma unroll
    for (int d = 8; d < kLanes; d <<= 1) y = op(y, __shfl_xor(y, d));
    if ((threadIdx.x & 63) < 8) red[slot][wave][q8] = y;
  };
  auto gathered = [&](int slot, auto op) {
    return op(op(red[slot][0][q8], red[slot][1][q8]), op(red[slot][2][q8], red[slot][3][q8]));
  };
  auto larger = [](float y, float z) { return fmaxf(y, z); };
  auto plus = [](float y, float z) { return y + z; };
  float mx = kNegInf;
#pragma unroll
  for (int i = 0; i < kAttendGrid / 32; ++i) mx = fmaxf(mx, ml[i].x);
  spread(mx, 0, larger);
  __syncthreads();
  mx = gathered(0, larger);
  float sum = 0.0f, rsum = 0.0f;
#pragma unroll
  for (int i = 0; i < kAttendGrid / 32; ++i) {
    const int k = piece + 32 * i;
    if (k >= sp.parts) break;
    const float e = ml[i].x == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ml[i].x - mx);
    weight[k][q8] = e;
    sum += ml[i].y * e;
    rsum += ml[i].z * e;
  }
  spread(sum, 1, plus);
  spread(rsum, 2, plus);
  __syncthreads();
  sum = gathered(1, plus);
  rsum = gathered(2, plus);
  f32x4 a[W] = {};
  auto add = [&](f32x4& to, const f32x4& y, float e) {
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = __builtin_fmaf(y[i], e, to[i]);
  };
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (i < sp.parts)
#pragma unroll
      for (int w = 0; w < W; ++w) add(a[w], v[i][w], weight[i][q8]);
#pragma unroll 4
  for (int k = P; k < sp.parts; ++k) {
    const float* const part = src + place(k) * kDim;
#pragma unroll
    for (int w = 0; w < W; ++w) add(a[w], *(const f32x4*)(part + 256 * w), weight[k][q8]);
  }
  const int32_t m = m0 + q8;
  if (m >= s.n * p.heads) return;
  const int32_t tok = (int32_t)udiv_magic((uint32_t)m, p.head_div.m, p.head_div.sh1, p.head_div.sh2);
  const int32_t head = m - tok * p.heads;
  const Final fin = finish(p.sink != nullptr ? p.sink[head] * kLog2e : kNegInf, mx, sum, rsum);
  uint16_t* const op = p.out + (int64_t)(s.first + tok) * p.out_stride + (int64_t)head * p.out_hstride;
#pragma unroll
  for (int w = 0; w < W; ++w)
    *(u32x2*)(op + 128 * (w0 + w) + 4 * piece) =
        u32x2{pack_bf16(a[w][0] * fin.f, a[w][1] * fin.f), pack_bf16(a[w][2] * fin.f, a[w][3] * fin.f)};
  if (p.lse != nullptr && w0 == 0 && piece == 0)
    p.lse[(int64_t)(s.first + tok) * p.heads + head] = fin.lse;
}

template <int L>
hipError_t attend(const AttendParams& p, int qblocks, hipStream_t stream) {
  const dim3 grid(kAttendGrid), block(kAttendBlock);
  const bool run = p.cache.page_bits >= 3;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, p);
    return hipGetLastError();
  };
  switch (qblocks) {
    case 1: return run ? go(attend_kernel<L, 1, true>) : go(attend_kernel<L, 1, false>);
    case 2: return run ? go(attend_kernel<L, 2, true>) : go(attend_kernel<L, 2, false>);
    default: return go(attend_wide_kernel<L>);
  }
}

}  // namespace

hipError_t launch_attend(const AttendParams& p, int qblocks, hipStream_t stream) {
  const int qt = 32 * qblocks, nt = 128 / qblocks;
  hipError_t e = hipSuccess;
  if (p.plan_units == 0) {
    hipLaunchKernelGGL(attend_plan_kernel, dim3(1), dim3(kPlanBlock), 0, stream, p, qt, nt);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  switch (p.cache.layout) {
    case kV41: e = attend<kV41>(p, qblocks, stream); break;
    case kV41Fp4: e = attend<kV41Fp4>(p, qblocks, stream); break;
    default: e = attend<kV4>(p, qblocks, stream); break;
  }
  if (e != hipSuccess) return e;
  // an entry per unit (plan_units), or per unit that is cut: one holds at least
  // one boundary between two workgroups
  const int64_t splits = p.plan_units > 0 ? (int64_t)p.num_slots * p.plan_units
                                          : min(p.units_max, (int64_t)kAttendGrid - 1);
  hipLaunchKernelGGL(attend_join_kernel, dim3((unsigned)splits, (unsigned)(qt / 8), 4 / kJoinWaves),
                     dim3(256), 0, stream, p, qt);
  return hipGetLastError();
}

}  // namespace kvc
