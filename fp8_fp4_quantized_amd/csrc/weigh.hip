// weigh.hip -- attention weight that cached rows collect (gfx950): for every row
// r of a slot, over the (token, head) pairs m of the slot that see it,
//   sum_m 2^(s_mr - lse_m),   s_mr = scale * log2(e) * (q_m . x_r),
// added to decay times what the row had.  lse is the attention's, so a pair's
// weights over its rows sum to 1 (less with a sink).
//
// Scores are products of matrix instructions with the queries as rows and the
// cached rows as columns of the result: a lane then holds 16 scores of one
// cached row, and the sum over the queries stays in its registers.  A lane reads
// the codes of its row straight from the page into the operand's place (dims in
// the order the codes come in; the queries are read from LDS in the same order),
// so pages of any size are alike and nothing of a row passes through LDS.
//
// What bounds it: a (query, row) pair is 1,024 flops, half of the attention's, and a
// row 288 to 584 bytes; at 1.5 PFLOP/s and 5.2 TB/s the two take the same time at 152
// queries a slot for V41, 83 for V41_FP4, 168 for V4.  Slots of few queries are bound by
// HBM: one token of 64 requests over V41 rows 70 us with 32 heads and 77 with 64 (4.6 and
// 4.2 TB/s), 128 chains of 4 with 16 heads over V4 rows 83 (4.3 TB/s); over V41_FP4 rows
// with 64 heads 57 us (2.9 TB/s), where the expansion, the products and the sums of
// half as many bytes share the time.  Slots of many are bound by the matrix units: a
// prompt of 8,192 tokens with 128 heads 3.7 to 3.9 ms (1.13 to 1.19 PFLOP/s; the same loop
// with products alone reaches 1.55 at the clock that the card holds under them), 16
// prompts of some 2,000 tokens with 32 heads over V41_FP4 rows pooled by two 0.71 to
// 0.77 ms, where 24% more pairs are multiplied than any token sees (3% for the prompt of
// 8,192): a block of 256 rows meets every token that sees its first.
#include <algorithm>

#include "launch_evict.hpp"
#include "row_ops.hpp"

namespace kvc {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

typedef const __attribute__((address_space(3))) uint8_t* lds_cptr;
typedef __attribute__((address_space(3))) uint8_t* lds_ptr;

constexpr float kNegInf = -__builtin_inff();

// tokens of slot b, the position of its first one and the rows they may see; n =
// 0 for a slot that has none or is skipped
struct SlotTokens {
  int32_t first, n, pos, rows;
};
__device__ __forceinline__ SlotTokens slot_tokens(const WeighParams& p, int b, int32_t* bad) {
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
  // row indices stay in int32
  if (s.n > 0 && (int64_t)s.pos + s.n > 0x7FFFFFFF - 256) {
    s.n = 0;
    *bad |= kStPosRange;
  }
  s.rows = s.n > 0 ? (s.pos + s.n) >> (p.ratio - 1) : 0;
  // rows past the table or the weights' row are left out
  const int64_t most = min(p.pt_width << p.cache.page_bits, p.w_width);
  if (s.rows > most) {
    s.rows = (int32_t)most;
    *bad |= kStPtRange;
  }
  return s;
}

// first token of the slot that sees row r
__device__ __forceinline__ int32_t first_token(const WeighParams& p, const SlotTokens& s, int32_t r) {
  if (p.tree != nullptr) return 0;
  const int64_t t = (int64_t)(r + 1) * p.ratio - 1 - s.pos;
  return t > 0 ? (int32_t)t : 0;
}

// rows below which every token of the slot sees all
__device__ __forceinline__ int32_t first_limit(const WeighParams& p, const SlotTokens& s) {
  return p.tree != nullptr ? s.pos : (s.pos + 1) >> (p.ratio - 1);
}

// ------------------------------------------------------------------ a row
// The codes of a lane's row, its half of each 64 (FP4) or 32 dims: lane l has
// row l % 32 of the wave's and half h = l / 32.  Step j of the product (16 dims,
// 8 a half) takes the dims of chunk(j) + 8-dim chunks of the half:
//   V41      dims 32 (j / 2) + 16 h + 8 (j % 2): load j / 2, scale byte j / 2
//   V41_FP4  dims 64 (j / 4) + 32 h + 8 (j % 4): load j / 4, scale byte 4 (j / 4) + 2 h + j % 4 / 2
//   V4       as V41 (scale byte j / 4) up to j = 27, then rope dims 448 + 16 (j - 28) + 8 h
template <int L> struct CodesShape;
template <> struct CodesShape<kV41> { static constexpr int kLoads = 16, kScales = 4; };
template <> struct CodesShape<kV41Fp4> { static constexpr int kLoads = 8, kScales = 8; };
template <> struct CodesShape<kV4> { static constexpr int kLoads = 18, kScales = 2; };

template <int L>
struct Codes {
  static constexpr int N = CodesShape<L>::kLoads;
  u32x4 code[N];
  uint32_t scale[CodesShape<L>::kScales];

  // data: the row's data part + 16 h; scale parts whole
  __device__ __forceinline__ void load_code(const uint8_t* data, int i) { code[i] = *(const u32x4*)(data + 32 * i); }
  __device__ __forceinline__ void load_scale(const uint8_t* sc) {
    if constexpr (L == kV4) {
      const u32x2 v = *(const u32x2*)sc;
      scale[0] = v.x, scale[1] = v.y;
    } else {
#pragma unroll
      for (int k = 0; k < CodesShape<L>::kScales / 4; ++k) {
        const u32x4 v = *(const u32x4*)(sc + 16 * k);
        scale[4 * k] = v.x, scale[4 * k + 1] = v.y, scale[4 * k + 2] = v.z, scale[4 * k + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void take_scale(const Codes& of) {
#pragma unroll
    for (int k = 0; k < CodesShape<L>::kScales; ++k) scale[k] = of.scale[k];
  }
  // load of step j (of its last one, the code is done with)
  static constexpr int load_of(int j) { return L == kV41Fp4 ? j >> 2 : L == kV4 && j >= 28 ? j - 14 : j >> 1; }
  static constexpr bool last_of(int j) { return L == kV41Fp4 ? (j & 3) == 3 : L == kV4 && j >= 28 ? true : (j & 1) != 0; }
  __device__ __forceinline__ bf16x8 expand(int j, int h) const {
    uint4 v;
    if constexpr (L == kV41Fp4) {
      const uint32_t pair = scale[j >> 2] >> (16 * h);
      v = dq_fp4x8(code[j >> 2][j & 3], (j & 2) ? pair >> 8 & 0xFFu : pair & 0xFFu);
    } else if (L == kV4 && j >= 28) {
      const u32x4 c = code[j - 14];
      v = make_uint4(c.x, c.y, c.z, c.w);
    } else {
      const int g = L == kV4 ? j >> 2 : j >> 1;
      const u32x4 c = code[j >> 1];
      v = dq_fp8x8((j & 1) ? make_uint2(c.z, c.w) : make_uint2(c.x, c.y), scale[g >> 2] >> (8 * (g & 3)) & 0xFFu);
    }
    return __builtin_bit_cast(bf16x8, u32x4{v.x, v.y, v.z, v.w});
  }
  // V41_FP4: 8 dims of step j as fp16.  The magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 have
  // no low byte in fp16, so their high bytes are looked up four at a time (v_perm_b32
  // takes bytes of an 8-byte table), the signs set, and the 8 products with the scale
  // are exact: at most 2,688, no less than 2^-10, 6 significant bits.  16 instructions
  // and a few a group where the conversions to fp32 and bf16 take 19, six of them slow.
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ f16x8 expand_f16(uint32_t w, f16x2 s) {
    const uint32_t even = __builtin_amdgcn_perm(0x46444240u, 0x3E3C3800u, w & 0x07070707u) | (w << 4 & 0x80808080u);
    const uint32_t odd = __builtin_amdgcn_perm(0x46444240u, 0x3E3C3800u, w >> 4 & 0x07070707u) | (w & 0x80808080u);
    u32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t pair = __builtin_amdgcn_perm(odd, even, 0x040C000Cu + 0x01000100u * k);
      v[k] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, pair) * s);
    }
    return __builtin_bit_cast(f16x8, v);
  }
  // the scales of step j's load, of its two groups
  __device__ __forceinline__ f16x2 scales_f16(int j, int h) const {
    return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)(scale[j >> 2] >> (16 * h)), 1.0f, false));
  }
  // 8-dim chunk of step j in a row of queries: that of half 0, and how far half 1 is
  static constexpr int chunk(int j) {
    return L == kV41Fp4 ? 8 * (j >> 2) + (j & 3) : L == kV4 && j >= 28 ? 56 + 2 * (j - 28) : 4 * (j >> 1) + (j & 1);
  }
  static constexpr int half_chunks(int j) { return L == kV41Fp4 ? 4 : L == kV4 && j >= 28 ? 1 : 2; }
};

// where a lane's row lies; a row that is none is read at row 0 of page 0
struct Place {
  const uint8_t* data;
  const uint8_t* scale;
  bool ok;
};
template <int L>
__device__ __forceinline__ Place place_of(const WeighParams& p, int64_t b, int32_t r, int32_t rows) {
  Place a;
  const int pb = p.cache.page_bits;
  int32_t page = 0;
  a.ok = (uint32_t)r < (uint32_t)rows;       // (a block past the last one may pass 2^31)
  if (a.ok) {
    page = p.page_table[b * p.pt_stride + (r >> pb)];
    if (page < 0 || page >= p.cache.num_pages) {
      a.ok = false;
      page = 0;
      if (p.status != nullptr) atomicOr(p.status, kStPageRange);
    }
  }
  const int64_t in = a.ok ? r & ((1 << pb) - 1) : 0;
  const uint8_t* base = p.cache.base + page * p.cache.page_stride;
  a.data = base + in * LayoutTraits<L>::kData + 16 * (lane_id() >> 5);
  a.scale = base + ((int64_t)LayoutTraits<L>::kData << pb) + in * LayoutTraits<L>::kScale;
  return a;
}

// The weight of row r after the call: decay times what it had, and its sum.  A row
// that this call's tokens complete begins at 0; a row that is not finite (its sum is
// not either) collects nothing.
__device__ __forceinline__ float old_weight(const WeighParams& p, int64_t b, const SlotTokens& s, int32_t r) {
  return p.prev != nullptr && r < s.pos >> (p.ratio - 1) ? p.prev[b * p.prev_stride + r] : 0.0f;
}
__device__ __forceinline__ void put_weight(const WeighParams& p, int64_t b, int32_t r, float old, float sum) {
  if (!(sum < __builtin_inff())) sum = 0.0f;
  p.weights[b * p.w_stride + r] = __builtin_fmaf(p.decay, old, sum);
}

__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ------------------------------------------------------------------ queries
// 32 queries of a slot in LDS: row m's 16-byte chunk c at place c ^ (m % 16) of
// its 1024 bytes (16 consecutive rows' chunks then lie in all banks), and of each
// query -lse, the rows below which all are seen, and a tree's mask.  A query past
// the end, or one whose lse is not finite (it has no rows, or no answer), gives
// nothing and has -lse = -inf.
struct QueryRows {
  float neg_lse[32];
  float factor[32];            // (few queries of FP4 rows) what their scores are multiplied by
  int32_t limit[32];
  // a tree: which drafted rows it sees, 32 a word, then a word for the rows of the
  // context and one for those past the drafts
  __attribute__((aligned(16))) uint32_t words[32][4];
};

// tree mask of a token
__device__ __forceinline__ uint64_t mask_of(const WeighParams& p, int64_t b, const SlotTokens& s, int32_t tok) {
  const uint64_t m = p.tree[b * p.draft_len + tok];
  return s.n < 64 ? m & ((uint64_t(1) << s.n) - 1) : m;
}

// A lane's query m of the slot's flat (token, head) list, which ends at `end`: where
// it lies (one past the end: where the last one does), and what is known of it.
// lse is as it is in memory, waited for where put is called.
struct LaneQuery {
  const uint16_t* at;
  float lse;
  int32_t token, limit;
  int64_t entry;               // of lse
  uint64_t mask;
  bool real;

  __device__ __forceinline__ void locate(const WeighParams& p, const SlotTokens& s, int32_t m, int32_t end) {
    real = m < end;
    const uint32_t n = (uint32_t)min(m, end - 1);
    token = (int32_t)udiv_magic(n, p.head_div.m, p.head_div.sh1, p.head_div.sh2);
    const uint32_t head = n - (uint32_t)token * (uint32_t)p.heads, row = (uint32_t)(s.first + token);
    // (strides are below 2^31)
    at = p.q + ((uint64_t)row * (uint32_t)p.q_stride + (uint64_t)head * (uint32_t)p.q_hstride);
    entry = (uint64_t)row * (uint32_t)p.heads + head;
    limit = p.tree != nullptr ? s.pos : (s.pos + token + 1) >> (p.ratio - 1);
  }
  // masks: whether a tree's masks matter (rows of drafted tokens are among those at hand)
  __device__ __forceinline__ void fetch(const WeighParams& p, int64_t b, const SlotTokens& s, bool masks) {
    lse = p.lse[entry];
    mask = masks ? mask_of(p, b, s, token) : 0;
  }
  __device__ __forceinline__ float neg_lse() const {
    return real && __builtin_fabsf(lse) < __builtin_inff() ? -lse : kNegInf;
  }
  __device__ __forceinline__ void put(QueryRows& info, int m) const {
    const float v = neg_lse();
    info.neg_lse[m] = v;
    info.limit[m] = v == kNegInf ? 0 : limit;
    *(u32x4*)info.words[m] = v == kNegInf ? u32x4{0, 0, 0, 0} : u32x4{(uint32_t)mask, (uint32_t)(mask >> 32), ~0u, 0};
  }
};

// 8 queries of a wave on their way to LDS, 8 lanes each: load i takes their i-th 128
// bytes.  m: the lane's query among those staged (8 * wave + lane / 8 + a multiple of 32).
struct Staged {
  u32x4 v[8];
  LaneQuery q;

  __device__ __forceinline__ void load(int i) {
    typedef const __attribute__((address_space(1))) u32x4* vec;
    v[i] = *(vec)((uint64_t)(uintptr_t)q.at + 128 * i + 16 * (lane_id() & 7));
  }
  // The query in fp16, times the power of two that brings its greatest value to
  // [2^14, 2^15); returns the power's inverse.  Exact for values down to 2^-31 of the
  // greatest; what is less is off by 2^-40 of that at the most, below the rounding of
  // an fp32 sum.  (The power is 2^126 at the most, for a greatest value below 2^-112; the
  // least, 2^-113, and the inverses of both are fp32 numbers.)
  __device__ __forceinline__ float to_f16() {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, absmax_bf16x8(make_uint4(v[i].x, v[i].y, v[i].z, v[i].w)));
    top = group_max_u32<8>(top);
    const int up = min(127 + 14 - (int)(top >> 7), 126);
    const float by = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = __builtin_bit_cast(uint16_t, (_Float16)(bf16_lo(v[i][k]) * by));
        const uint32_t hi = __builtin_bit_cast(uint16_t, (_Float16)(bf16_hi(v[i][k]) * by));
        v[i][k] = lo | hi << 16;
      }
    }
    return __uint_as_float((uint32_t)(127 - up) << 23);
  }
  static __device__ __forceinline__ uint32_t place(int m) {
    return m * 1024 + 16 * ((lane_id() & 7) ^ (m & 15));
  }
  __device__ __forceinline__ void store(lds_ptr rows, int m, int i) const {
    *(__attribute__((address_space(3))) u32x4*)(rows + (place(m) ^ (128 * (i & 1))) + 256 * (i >> 1)) = v[i];
  }
  __device__ __forceinline__ void put(QueryRows& info, int m) const {
    if ((lane_id() & 7) == 0) q.put(info, m);
  }
};

// The word and bit of a query's that say whether it sees row r; base: the first
// drafted row
struct TreeBit {
  int32_t word, bit;
  __device__ __forceinline__ TreeBit(int32_t r, int32_t base) {
    const uint32_t x = (uint32_t)(r - base);
    word = r < base ? 2 : x < 64u ? (int32_t)(x >> 5) : 3;
    bit = r < base ? 0 : (int32_t)(x & 31u);
  }
  // v where it is seen, else 0 (whatever v is)
  __device__ __forceinline__ float kept(float v, const QueryRows& q, int m) const {
    const int32_t all = __builtin_amdgcn_sbfe((int)q.words[m][word], bit, 1);
    return __uint_as_float(__float_as_uint(v) & (uint32_t)all);
  }
};

// wait states from a last product to what reads, or overwrites, its result
__device__ __forceinline__ void scores_done(f32x16& sc) { asm("s_nop 15" : "+v"(sc)); }

// Adds a lane's 16 weights of a 32 x 32 result to v.  masked: some of the
// queries may not see some of the rows, or give nothing.
// OWN: each query has its own factor.
template <bool OWN>
__device__ __forceinline__ float add_weights(float v, const f32x16& s, float scale, const QueryRows& q, int h,
                                             bool masked, int32_t r, bool tree, int32_t base) {
  const TreeBit of(r, base);
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const f32x4 nl = *(const f32x4*)&q.neg_lse[8 * a + 4 * h];
    f32x4 factor = f32x4{scale, scale, scale, scale};
    if constexpr (OWN) factor = *(const f32x4*)&q.factor[8 * a + 4 * h];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * a + i], factor[i], nl[i]));
      if (masked) {
        const int m = 8 * a + 4 * h + i;
        w = tree ? of.kept(w, q, m) : r < q.limit[m] ? w : 0.0f;
      }
      v += w;
    }
  }
  return v;
}

// ------------------------------------------------------------------ batch
// Sums over the slots in LDS: of a call's blocks of rows, or of its cost.
template <int BLOCK>
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t* buf, int64_t* total) {
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
  for (int w = 0; w < BLOCK / kLanes; ++w) {
    if (w == wave) x += t;
    t += buf[w];
  }
  *total = t;
  return x;
}

// last slot whose sum before it is <= at (slots that add nothing share the start
// of the next one)
template <typename T>
__device__ __forceinline__ int slot_at(const T* before, int n, T at) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= at) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------------ few queries
// Slots of up to 32 NC queries each, 128 at the most: they stay in LDS while 8 waves,
// two to a SIMD, go over the slot's rows, 32 at a time.  Measured beside the kernel for
// many queries, one token of 64 requests with 128 heads: V41 111 us and 195, V41_FP4 98
// and 177; of one request of 1,000 rows 12 and 24.
constexpr int kFewBlock = 512;
constexpr int kFewWaves = kFewBlock / kLanes;
constexpr int kFewGrid = 256;

// A slot's begin, its queries brought to LDS, as the blocks that take the same time
// (64 decodes: 8 blocks 63.1 us, 16 62.7, 24 61.8, 40 63.9)
constexpr uint32_t kSlotBlocks = 16;
__device__ __forceinline__ uint32_t few_cost(int32_t rows) {
  return rows > 0 ? (uint32_t)((rows + 31) >> 5) + kSlotBlocks : 0;
}

template <int NC> constexpr int kReadAheadOf = NC > 2 ? 2 : 3;   // (what registers are left)

template <int L, int NC, int SLOTS>
__global__ __launch_bounds__(kFewBlock) void weigh_few_kernel(WeighParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t rows[NC * 32 * 1024];
  __shared__ QueryRows info[NC];
  constexpr bool kF16 = L == kV41Fp4;          // (rows and queries in fp16)
  constexpr int kReadAhead = kReadAheadOf<NC>;
  // cost of the slots before each second one
  __shared__ uint32_t before[SLOTS / 2];
  __shared__ int64_t buf[kFewWaves];
  const int S = p.num_slots, tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
  const int h = lane >> 5;
  int32_t bad = 0;
  int64_t carry = 0;
  for (int b0 = 0; b0 < S; b0 += 2 * kFewBlock) {
    const int b = b0 + 2 * tid;
    int64_t n0 = 0, n1 = 0, total;
    if (b < S) n0 = few_cost(slot_tokens(p, b, &bad).rows);
    if (b + 1 < S) n1 = few_cost(slot_tokens(p, b + 1, &bad).rows);
    const int64_t end = block_scan64<kFewBlock>(n0 + n1, buf, &total) + carry;
    if (b < S) before[b >> 1] = (uint32_t)(end - n0 - n1);
    carry += total;
  }
  if (blockIdx.x == 0 && bad != 0 && p.status != nullptr) atomicOr(p.status, bad);
  __syncthreads();
  const uint32_t all = (uint32_t)carry;
  const uint32_t quota = (all + gridDim.x - 1) / gridDim.x;
  uint32_t at = min(all, quota * blockIdx.x);
  const uint32_t to = min(all, at + quota);
  while (at < to) {
    // the slot at that place
    int b = 2 * slot_at(before, (S + 1) >> 1, at);
    uint32_t first = before[b >> 1];
    int32_t none = 0;
    SlotTokens s = slot_tokens(p, b, &none);
    if (at - first >= few_cost(s.rows)) {
      first += few_cost(s.rows);
      ++b;
      s = slot_tokens(p, b, &none);
    }
    b = uniform(b);
    first = uniform((int32_t)first);
    s = SlotTokens{uniform(s.first), uniform(s.n), uniform(s.pos), uniform(s.rows)};
    // its blocks from k0 to k1
    const uint32_t k0 = max(at, first + kSlotBlocks) - first - kSlotBlocks;
    const uint32_t end = min(to, first + few_cost(s.rows));
    const uint32_t k1 = max(end, first + kSlotBlocks) - first - kSlotBlocks;
    at = end;
    if (k0 >= k1) continue;
    // its queries
    const int32_t nq = s.n * p.heads;
    __syncthreads();
    for (int m0 = 8 * wave; m0 < 32 * NC; m0 += 8 * kFewWaves) {
      Staged g;
      const int m = m0 + (lane >> 3);
      g.q.locate(p, s, m, nq);
      g.q.fetch(p, b, s, p.tree != nullptr);
#pragma unroll
      for (int i = 0; i < 8; ++i) g.load(i);
      g.put(info[m0 >> 5], m & 31);
      // (zeros in place of a query that gives nothing: its weights are then 0 of
      // themselves)
      const bool gives = g.q.neg_lse() != kNegInf;
      if constexpr (kF16) {
        const float back = g.to_f16();
        if ((lane & 7) == 0) info[m0 >> 5].factor[m & 31] = p.scale_log2 * back;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!gives) g.v[i] = u32x4{0, 0, 0, 0};
        g.store((lds_ptr)rows, m, i);
      }
    }
    __syncthreads();
    // its rows
    const int32_t clear = first_limit(p, s);
    // (a block's codes take the place of the one before as its products are done)
    uint32_t k = k0 + wave;
    if (k < k1) {
      auto row_of = [&](uint32_t block) { return (int32_t)(32 * block) + (lane & 31); };
      Place here = place_of<L>(p, b, row_of(k), s.rows);
      Codes<L> c;
#pragma unroll
      for (int i = 0; i < Codes<L>::N; ++i) c.load_code(here.data, i);
      c.load_scale(here.scale);
      Place next = place_of<L>(p, b, row_of(k + kFewWaves), min(s.rows, (int32_t)(32 * k1)));
      for (; k < k1; k += kFewWaves) {
        // (the queries' fragments are read again for every block: kept over the
        // loop they would not fit)
        asm volatile("" ::: "memory");
        const int row_base = (lane & 31) * 1024, low = lane & 15;
        const int32_t r = row_of(k);
        const float old = old_weight(p, b, s, min(r, s.rows - 1));
        Codes<L> after;                       // its scales
        after.load_scale(next.scale);
        const Place then = place_of<L>(p, b, row_of(k + 2 * kFewWaves), min(s.rows, (int32_t)(32 * k1)));
        f32x16 acc[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) acc[n] = f32x16{};
        // (fragments are read kReadAhead steps and a step's dims expanded one before their
        // products, which they share the time with)
        typename Codes<L>::f16x2 pair = {};
        auto dims_of = [&](int j) {
          if constexpr (kF16) {
            if ((j & 3) == 0) pair = c.scales_f16(j, h);
            const _Float16 g = pair[j >> 1 & 1];
            return __builtin_bit_cast(bf16x8, Codes<L>::expand_f16(c.code[j >> 2][j & 3], typename Codes<L>::f16x2{g, g}));
          } else {
            return c.expand(j, h);
          }
        };
        bf16x8 q[kReadAhead][NC];
        auto read = [&](int j) {
          const uint32_t at_row = row_base + 16 * ((Codes<L>::chunk(j) + Codes<L>::half_chunks(j) * h) ^ low);
#pragma unroll
          for (int n = 0; n < NC; ++n) q[j % kReadAhead][n] = *(const bf16x8*)(rows + n * 32 * 1024 + at_row);
        };
#pragma unroll
        for (int j = 0; j < kReadAhead; ++j) read(j);
        bf16x8 x = dims_of(0);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const bf16x8 a = q[j % kReadAhead][n];
            if constexpr (kF16)
              acc[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                              __builtin_bit_cast(f16x8, x), acc[n], 0, 0, 0);
            else
              acc[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, x, acc[n], 0, 0, 0);
          }
          if (j + kReadAhead < 32) read(j + kReadAhead);
          if (j + 1 < 32) x = dims_of(j + 1);
          // (the loads of a row's 128 bytes together: a line is then fetched once)
          constexpr int kLast = Codes<L>::N - 1;
          const int i = Codes<L>::load_of(j);
          if (Codes<L>::last_of(j) && ((i & 3) == 3 || i == kLast)) {
#pragma unroll
            for (int t = i & ~3; t <= i; ++t) c.load_code(next.data, t);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) scores_done(acc[n]);
        const bool masked = (int32_t)(32 * k) + 32 > clear;
        float v = 0.0f;
#pragma unroll
        for (int n = 0; n < NC; ++n)
          v = masked ? add_weights<kF16>(v, acc[n], p.scale_log2, info[n], h, true, r, p.tree != nullptr, s.pos)
                     : add_weights<kF16>(v, acc[n], p.scale_log2, info[n], h, false, r, false, 0);
        v = sum_halves(v);
        if (lane < 32 && r < s.rows) put_weight(p, b, r, old, here.ok ? v : 0.0f);
        here = next;
        next = then;
        c.take_scale(after);
      }
    }
  }
}

// ------------------------------------------------------------------ many queries
// Blocks of 256 rows, 64 a wave, whose operands stay in registers while the
// queries that see them pass through LDS, 32 at a time.  A slot's tokens are cut
// into segments of 2^cut tokens; a part is a segment's queries with one of the
// blocks that they see.  Parts are numbered segment by segment, an eighth of them
// goes to the workgroups of each XCD, which take them in turn: those that run at
// the same time share a segment, and its queries come from their L2 (a prompt of
// 8,192 tokens with 128 heads is 1 GB of queries, each seen by 16 blocks on
// average).  The sums of a slot of several segments go to the workspace, and
// weigh_join_kernel adds them in order.
constexpr int kManyBlock = 256;
constexpr int kManyRowBits = 8;
static_assert(kWeighRows == 1 << kManyRowBits, "rows of a block");
constexpr int kXcds = 8;

__device__ __forceinline__ int32_t blocks_of(const SlotTokens& s) {
  return (int32_t)(((int64_t)s.rows + kWeighRows - 1) >> kManyRowBits);
}
__device__ __forceinline__ int32_t segments_of(const SlotTokens& s, int cut) {
  return (int32_t)(((int64_t)s.n + (int64_t(1) << cut) - 1) >> cut);
}

// (token, head) pairs of all blocks of a slot with the tokens that see their
// first row: those from first_token on, which is 0 or grows by rows * ratio a block
__device__ __forceinline__ int64_t work_of(const WeighParams& p, const SlotTokens& s) {
  const int64_t k = blocks_of(s);
  int64_t tokens = s.n * k;
  if (p.tree == nullptr) {
    const int step = kManyRowBits + p.ratio - 1;
    const int64_t c = p.ratio - 1 - (int64_t)s.pos;            // first_token of block i: (i << step) + c, or 0
    const int64_t i1 = c > 0 ? 0 : (-c >> step) + 1;
    if (k > i1) tokens -= (k - i1) * (((i1 + k - 1) << step) + 2 * c) / 2;
  }
  return tokens * p.heads;
}

// sum of i >> d over i < n
__device__ __forceinline__ int64_t sum_shifted(int64_t n, int d) {
  const int64_t q = n >> d, r = n & ((int64_t(1) << d) - 1);
  return (q * (q - 1) / 2 << d) + r * q;
}

// Parts of the first g segments of a slot: the blocks that their last tokens see.
// The last token of segment i sees (pos + (i + 1) 2^cut) >> (ratio - 1) rows, in
// (y + i 2^cut) >> s blocks, y and s as below; the slot's last segment, and a
// segment past the rows there are, see all of them.
__device__ __forceinline__ int64_t parts_before(const WeighParams& p, const SlotTokens& s, int cut, int64_t g) {
  const int64_t all = blocks_of(s);
  if (p.tree != nullptr) return g * all;
  const int64_t G = segments_of(s, cut), few = min(g, G - 1);
  const int sh = kManyRowBits + p.ratio - 1;
  const int64_t y = (int64_t)s.pos + (int64_t(1) << cut) + ((int64_t)(kWeighRows - 1) << (p.ratio - 1));
  // segments that see fewer than all
  const int64_t reach = (all << sh) - y;      // y + i 2^cut < all 2^s
  const int64_t part = min(few, reach > 0 ? (reach + (int64_t(1) << cut) - 1) >> cut : 0);
  const int64_t sum = cut >= sh ? part * (y >> sh) + ((part * (part - 1) / 2) << (cut - sh))
                                : sum_shifted((y >> cut) + part, sh - cut) - sum_shifted(y >> cut, sh - cut);
  return sum + (g - part) * all;
}
__device__ __forceinline__ int64_t parts_of(const WeighParams& p, const SlotTokens& s, int cut) {
  return s.n > 0 ? parts_before(p, s, cut, segments_of(s, cut)) : 0;
}

// The first cut tried: segments of `share` queries, a sixteenth of a workgroup's
// share of the work, but 2,048 or the whole share where that is less, and 128 at the
// least (4 chunks; fewer would not pay for the block's begin).  Measured for the
// prompt of 8,192 tokens and the 16 of some 2,000, us: a 32nd and 1,024 4,372 and 961, a
// 16th and 2,048 4,290 and 910, a 16th and 4,096 4,283 and 878, an 8th and 2,048 4,538
// and 905.  (Longer segments leave fewer parts to deal.)
__device__ __forceinline__ int first_cut(const WeighParams& p, int64_t work) {
  const int64_t each = (work + kWeighWorkgroups - 1) / kWeighWorkgroups;
  const int64_t share = max(max(each / 16, min(each, (int64_t)2048)), (int64_t)128);
  int cut = 0;
  while ((int64_t)p.heads << (cut + 1) <= share && cut < 30) ++cut;
  return cut;
}

// Sums over the slots before each second one: of their parts, and of those of
// them that go to the workspace.
template <int SLOTS>
struct Deal {
  uint32_t parts[SLOTS / 2], stored[SLOTS / 2];
};
// fills it for a cut; returns the totals to every thread
struct Totals {
  int64_t parts, stored;
};
template <int SLOTS>
__device__ __forceinline__ Totals deal_parts(const WeighParams& p, int cut, Deal<SLOTS>& d, int64_t* buf) {
  Totals t{0, 0};
  for (int b0 = 0; b0 < p.num_slots; b0 += 2 * kManyBlock) {
    const int b = b0 + 2 * (int)threadIdx.x;
    int64_t n = 0, m = 0, total;
    int32_t none = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (b + i >= p.num_slots) continue;
      const SlotTokens s = slot_tokens(p, b + i, &none);
      const int64_t parts = parts_of(p, s, cut);
      n += parts;
      m += segments_of(s, cut) > 1 ? parts : 0;
    }
    const int64_t ne = block_scan64<kManyBlock>(n, buf, &total) + t.parts;
    t.parts += total;
    const int64_t me = block_scan64<kManyBlock>(m, buf, &total) + t.stored;
    t.stored += total;
    if (b < p.num_slots) d.parts[b >> 1] = (uint32_t)(ne - n), d.stored[b >> 1] = (uint32_t)(me - m);
  }
  __syncthreads();
  return t;
}

// A part: its slot, segment and block, and its place in the workspace (-1: the
// slot has one segment).
struct Part {
  int b;
  SlotTokens s;
  int32_t g, k;
  int64_t stored;
};
template <int SLOTS>
__device__ __forceinline__ Part part_at(const WeighParams& p, const Deal<SLOTS>& d, int cut, uint32_t at) {
  Part x;
  x.b = 2 * slot_at(d.parts, (p.num_slots + 1) >> 1, at);
  int64_t in = at - d.parts[x.b >> 1], base = d.stored[x.b >> 1];
  int32_t none = 0;
  SlotTokens s = slot_tokens(p, x.b, &none);
  const int64_t mine = parts_of(p, s, cut);
  if (in >= mine) {
    in -= mine;
    if (segments_of(s, cut) > 1) base += mine;
    s = slot_tokens(p, ++x.b, &none);
  }
  x.b = uniform(x.b);
  x.s = SlotTokens{uniform(s.first), uniform(s.n), uniform(s.pos), uniform(s.rows)};
  const int32_t G = segments_of(x.s, cut);
  int32_t lo = 0, hi = G - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (parts_before(p, x.s, cut, mid) <= in) lo = mid;
    else hi = mid - 1;
  }
  x.g = uniform(lo);
  x.k = uniform((int32_t)(in - parts_before(p, x.s, cut, lo)));
  x.stored = G > 1 ? uniform64(base + in) : -1;
  return x;
}

// The products are written out so that the rows stay in the 256 accumulator
// registers and the scores in the vector registers their sums work in.  Their
// operands come from LDS and from registers that stay; a result that feeds the next
// product's C operand needs no wait.  The build reads the assembly for the wait
// states and stops where one is missing.
__device__ __forceinline__ void score_mfma(f32x16& sc, bf16x8 q, const bf16x8& x, bool first) {
  if (first) asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(sc) : "v"(q), "a"(x));
  else asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+&v"(sc) : "v"(q), "a"(x));
}

// 32 queries in LDS, as loads bring them there by themselves, 64 consecutive
// 16-byte places each: groups of 8 queries, of each its dims in pieces of 64, of
// each piece the 8 queries' 128 bytes.  Which query and chunk a place holds is the
// lane's choice of address: query m of the group is at row m ^ (group % 2), its chunk c
// of the piece at c ^ m, so that 16 consecutive queries' chunks lie in all banks.
constexpr int kChunkBytes = 32 * 1024;
struct Staging : LaneQuery {
  // piece I, from the lane's part of its query (8 dims at 8 * part) to the place `to` of
  // LDS, below 64 KB, + 1024 I
  template <int I>
  __device__ __forceinline__ void load(uint32_t to, int part) const {
    asm volatile("s_add_u32 m0, %0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to),
                 "v"(at + 8 * part + 64 * I), "n"(1024 * I)
                 : "memory", "m0", "scc");
  }
  __device__ __forceinline__ void load_all(uint32_t to, int part) const {
    load<0>(to, part), load<1>(to, part), load<2>(to, part), load<3>(to, part);
    load<4>(to, part), load<5>(to, part), load<6>(to, part), load<7>(to, part);
  }
  // all that was asked for is there
  __device__ __forceinline__ void arrive(QueryRows& info, int m) const {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if ((lane_id() & 7) == 0) put(info, m);
  }
};

// a lane's place in a staged chunk of step j's queries
template <int L>
__device__ __forceinline__ uint32_t query_at(int j, int lane) {
  const int c = Codes<L>::chunk(j), m = lane & 31;
  const uint32_t base = (m >> 3) * 8192 + ((m & 7) ^ (m >> 3 & 1)) * 128 +
                        16 * ((Codes<L>::half_chunks(j) * (lane >> 5)) ^ (m & 7));
  return (base ^ (16 * (c & 7))) + 1024 * (c >> 3);
}

constexpr int kAhead = 4;        // fragments of queries read ahead (3 and 6 measure the same, 8 2% slower)

// The scores of a chunk of 32 queries with the wave's 64 rows.  SUM 1: the weights
// of the chunk before (scores prev, queries of) are added up meanwhile, one a step,
// their three instructions a step apart; 2: those of rows below each query's own
// limit (r: the lane's first row); 3: those that a tree's queries see (base: the first
// drafted row).  beside(j) is done in step j.
template <int L, int SUM, typename Beside>
__device__ __forceinline__ void scores_of(f32x16 (&sc)[2], const bf16x8 (&x)[2][32], lds_cptr rows, int lane,
                                          const f32x16 (&prev)[2], const QueryRows& of, int32_t r, int32_t base,
                                          float scale, float (&sum)[2], Beside&& beside) {
  bf16x8 q[kAhead];
  float arg = 0.0f, w = 0.0f;
  const int h = lane >> 5;
  f32x4 nl[4];
  i32x4 lim[4];
  if constexpr (SUM > 0) {
#pragma unroll
    for (int a = 0; a < 4; ++a) nl[a] = *(const f32x4*)&of.neg_lse[8 * a + 4 * h];
  }
  if constexpr (SUM == 2) {
#pragma unroll
    for (int a = 0; a < 4; ++a) lim[a] = *(const i32x4*)&of.limit[8 * a + 4 * h];
  }
  // weight of step j: of scores prev[j % 2], element j / 2
  const TreeBit bit0(r, base), bit1(r + 32, base);
  auto kept = [&](float v, int j) {
    if constexpr (SUM == 2) return r + 32 * (j & 1) < lim[j >> 3][j >> 1 & 3] ? v : 0.0f;
    if constexpr (SUM == 3) return ((j & 1) ? bit1 : bit0).kept(v, of, 8 * (j >> 3) + 4 * h + (j >> 1 & 3));
    return v;
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) q[j] = *(const __attribute__((address_space(3))) bf16x8*)(rows + query_at<L>(j, lane));
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    score_mfma(sc[0], q[j % kAhead], x[0][j], j == 0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (SUM > 0) {
      if (j > 1) sum[j & 1] += kept(w, j - 2);
      if (j > 0) w = __builtin_amdgcn_exp2f(arg);
    }
    __builtin_amdgcn_sched_barrier(0);
    score_mfma(sc[1], q[j % kAhead], x[1][j], j == 0);
    __builtin_amdgcn_sched_barrier(0);
    if (j + kAhead < 32)
      q[j % kAhead] = *(const __attribute__((address_space(3))) bf16x8*)(rows + query_at<L>(j + kAhead, lane));
    if constexpr (SUM > 0) arg = __builtin_fmaf(prev[j & 1][j >> 1], scale, nl[j >> 3][j >> 1 & 3]);
    beside(j);
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (SUM > 0) {
    sum[0] += kept(w, 30);
    sum[1] += kept(__builtin_amdgcn_exp2f(arg), 31);
  }
  scores_done(sc[0]);
  scores_done(sc[1]);
}

// A sum with the rounding errors of its additions carried along (a slot's queries
// may be a million)
struct Total {
  float sum, low;
  __device__ __forceinline__ void add(float v) {
    const float y = v - low, t = sum + y;
    low = (t - sum) - y;
    sum = t;
  }
};

template <int L, int SLOTS>
__global__ __launch_bounds__(kManyBlock) void weigh_many_kernel(WeighParams p) {
  // (one object, the chunks at its begin)
  __shared__ struct {
    __attribute__((aligned(1024))) uint8_t rows[2][kChunkBytes];
    QueryRows info[3];
    Deal<SLOTS> deal;
    int64_t buf[kManyBlock / kLanes];
  } sh;
  QueryRows* const info = sh.info;
  const int S = p.num_slots, tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
  const int h = lane >> 5;
  int32_t bad = 0;
  int64_t work = 0;
  for (int b = tid; b < S; b += kManyBlock) work += work_of(p, slot_tokens(p, b, &bad));
  block_scan64<kManyBlock>(work, sh.buf, &work);
  if (blockIdx.x == 0 && bad != 0 && p.status != nullptr) atomicOr(p.status, bad);
  // (longer segments where there would be more parts than places for them)
  int cut = first_cut(p, uniform64(work));
  Totals all = deal_parts(p, cut, sh.deal, sh.buf);
  while (all.stored > kWeighParts) all = deal_parts(p, ++cut, sh.deal, sh.buf);
  if (blockIdx.x == 0 && tid == 0) p.head->cut = cut;
  const int64_t count = uniform64(all.parts);
  const uint32_t xcd = blockIdx.x % kXcds, to = (uint32_t)(count * (xcd + 1) / kXcds);
  for (uint32_t at = (uint32_t)(count * xcd / kXcds) + blockIdx.x / kXcds; at < to; at += kWeighWorkgroups / kXcds) {
    const Part blk = part_at(p, sh.deal, cut, at);
    const SlotTokens& s = blk.s;
    const int32_t ta = max(first_token(p, s, blk.k << kManyRowBits), blk.g << cut);
    const int32_t tb = (int32_t)min((int64_t)s.n, (int64_t)(blk.g + 1) << cut);
    const int32_t end = tb * p.heads;
    int32_t m0 = ta * p.heads;
    // the lane's query of a chunk, when they are staged, and its part of it
    const int mine = 8 * wave + ((lane >> 3) ^ (wave & 1)), part8 = (lane & 7) ^ (mine & 7);
    Staging g[2];
    g[0].locate(p, s, m0 + mine, end);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr)sh.rows[0] + 8192 * wave;
    g[0].load_all(lds0, part8);
    const bool masks = p.tree != nullptr && (int64_t)(blk.k + 1) << kManyRowBits > s.pos;
    g[0].fetch(p, blk.b, s, masks);
    g[1].locate(p, s, m0 + 32 + mine, end);
    // its rows
    const int32_t r0 = (blk.k << kManyRowBits) + 64 * wave;
    bf16x8 x[2][32];
    bool ok[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const Place pl = place_of<L>(p, blk.b, r0 + 32 * n + (lane & 31), s.rows);
      ok[n] = pl.ok;
      Codes<L> c;
#pragma unroll
      for (int i = 0; i < Codes<L>::N; ++i) c.load_code(pl.data, i);
      c.load_scale(pl.scale);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        x[n][j] = c.expand(j, h);
        asm volatile("" : "+a"(x[n][j]));     // (to stay there)
      }
    }
    g[0].arrive(info[0], mine);
    __syncthreads();
    // The queries, 32 a turn, the weights of a turn's scores added in the next one.
    // Where the queries of a chunk all see the same rows (those of a token's heads do),
    // a lane takes its sum or leaves it (`limit`); where they do not, each weight has
    // its own condition.
    Total total[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
    f32x16 sc[2][2];
    bool waiting = false, same = false;
    int32_t limit = 0;                        // of the chunk before, where `same`
    int now = 0;                              // of info's three
    auto add_chunk = [&](f32x16 (&of)[2], const QueryRows& q) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
        total[n].add(add_weights<false>(0.0f, of[n], p.scale_log2, q, h, true, r0 + 32 * n + (lane & 31), p.tree != nullptr,
                                 s.pos));
    };
    // (the running sums are added up in fp32 for 8 turns, then into the totals)
    float part[2] = {0.0f, 0.0f};
    int turns = 0;
    auto step = [&](f32x16 (&cur)[2], f32x16 (&prev)[2], lds_cptr here, uint32_t there, Staging& next, Staging& after) {
      const QueryRows& before = info[now == 0 ? 2 : now - 1];
      const int32_t mine_sees = info[now].limit[lane & 31];
      // the next chunk is asked for between the first products, the one after it
      // located between the last
      auto beside = [&](int j) {
        if (j == 0) next.load<0>(there, part8), next.load<1>(there, part8);
        if (j == 1) next.load<2>(there, part8), next.load<3>(there, part8);
        if (j == 2) next.load<4>(there, part8), next.load<5>(there, part8);
        if (j == 3) next.load<6>(there, part8), next.load<7>(there, part8);
        if (j == 4) next.fetch(p, blk.b, s, masks);
        if (j == 20) after.locate(p, s, m0 + 64 + mine, end);
      };
      float sum[2] = {0.0f, 0.0f};
      if (waiting && same) {
        scores_of<L, 1>(cur, x, here, lane, prev, before, 0, 0, p.scale_log2, sum, beside);
#pragma unroll
        for (int n = 0; n < 2; ++n) sum[n] = r0 + 32 * n + (lane & 31) < limit ? sum[n] : 0.0f;
      } else if (waiting && p.tree == nullptr) {
        scores_of<L, 2>(cur, x, here, lane, prev, before, r0 + (lane & 31), 0, p.scale_log2, sum, beside);
      } else if (waiting) {
        scores_of<L, 3>(cur, x, here, lane, prev, before, r0 + (lane & 31), s.pos, p.scale_log2, sum, beside);
      } else {
        scores_of<L, 0>(cur, x, here, lane, prev, before, 0, 0, 0.0f, sum, beside);
      }
      part[0] += sum[0];
      part[1] += sum[1];
      if ((++turns & 7) == 0) {
        total[0].add(part[0]);
        total[1].add(part[1]);
        part[0] = part[1] = 0.0f;
      }
      // (the rows of the wave, all below every limit, or cut by the same one)
      limit = uniform(mine_sees);
      same = __ballot(mine_sees != limit) == 0 && (p.tree == nullptr || r0 + 64 <= limit);
      if (__ballot(mine_sees < r0 + 64) == 0) same = true, limit = 0x7FFFFFFF;
      waiting = true;
      now = now == 2 ? 0 : now + 1;
      next.arrive(info[now], mine);
      __syncthreads();
      m0 += 32;
    };
    while (true) {
      step(sc[0], sc[1], (lds_cptr)sh.rows[0], lds0 + kChunkBytes, g[1], g[0]);
      if (m0 >= end) {
        add_chunk(sc[0], info[now == 0 ? 2 : now - 1]);
        break;
      }
      step(sc[1], sc[0], (lds_cptr)sh.rows[1], lds0, g[0], g[1]);
      if (m0 >= end) {
        add_chunk(sc[1], info[now == 0 ? 2 : now - 1]);
        break;
      }
    }
    total[0].add(part[0]);
    total[1].add(part[1]);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float both = sum_halves(total[n].sum), sum = ok[n] ? both : 0.0f;
      const int32_t r = r0 + 32 * n + (lane & 31);
      if (lane < 32) {
        if (blk.stored >= 0) p.parts[blk.stored * kWeighRows + 64 * wave + 32 * n + lane] = sum;
        else if (r < s.rows) put_weight(p, blk.b, r, old_weight(p, blk.b, s, r), sum);
      }
    }
    __syncthreads();                          // info and rows are free
  }
}

// The sums of the slots that have several segments: a workgroup a block of rows,
// its parts dealt to four groups of threads and added in order, with the errors of the
// additions carried along (a prompt of 2,500 tokens of 1,024 heads has 1,250 parts a row).
constexpr int kJoinBlock = 1024;
constexpr int kJoinGroups = kJoinBlock / kWeighRows;

template <int SLOTS>
__global__ __launch_bounds__(kJoinBlock) void weigh_join_kernel(WeighParams p) {
  __shared__ uint32_t blocks[SLOTS / 2], stored[SLOTS / 2];
  __shared__ int64_t buf[kJoinBlock / kLanes];
  __shared__ float sums[kJoinGroups][kWeighRows];
  __shared__ int32_t place[kJoinBlock];
  const int cut = uniform(p.head->cut), S = p.num_slots;
  int64_t count = 0, places = 0;
  int32_t none = 0;
  for (int b0 = 0; b0 < S; b0 += 2 * kJoinBlock) {
    const int b = b0 + 2 * (int)threadIdx.x;
    int64_t n = 0, m = 0, total;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (b + i >= S) continue;
      const SlotTokens s = slot_tokens(p, b + i, &none);
      if (segments_of(s, cut) > 1) n += blocks_of(s), m += parts_of(p, s, cut);
    }
    const int64_t ne = block_scan64<kJoinBlock>(n, buf, &total) + count;
    count += total;
    const int64_t me = block_scan64<kJoinBlock>(m, buf, &total) + places;
    places += total;
    if (b < S) blocks[b >> 1] = (uint32_t)(ne - n), stored[b >> 1] = (uint32_t)(me - m);
  }
  __syncthreads();
  const int row = threadIdx.x % kWeighRows, group = threadIdx.x / kWeighRows;
  for (uint32_t at = blockIdx.x; at < (uint32_t)count; at += gridDim.x) {
    int b = 2 * slot_at(blocks, (S + 1) >> 1, at);
    int64_t k = at - blocks[b >> 1], base = stored[b >> 1];
    SlotTokens s = slot_tokens(p, b, &none);
    const int64_t mine = segments_of(s, cut) > 1 ? blocks_of(s) : 0;
    if (k >= mine) {
      if (mine > 0) base += parts_of(p, s, cut);
      k -= mine;
      s = slot_tokens(p, ++b, &none);
    }
    // the block's parts: of the segments from the one of the first token that sees it
    const int32_t G = segments_of(s, cut), g0 = first_token(p, s, (int32_t)k << kManyRowBits) >> cut;
    Total v{0.0f, 0.0f};
    for (int32_t t0 = g0; t0 < G; t0 += kJoinBlock) {
      // their places, a thread each
      const int32_t mine_at = t0 + (int32_t)threadIdx.x, n = min(G - t0, kJoinBlock);
      __syncthreads();
      if (mine_at < G) place[threadIdx.x] = (int32_t)(base + parts_before(p, s, cut, mine_at) + k);
      __syncthreads();
#pragma unroll 8
      for (int32_t t = group; t < n; t += kJoinGroups) v.add(p.parts[(int64_t)place[t] * kWeighRows + row]);
    }
    sums[group][row] = v.sum;
    __syncthreads();
    const int32_t r = ((int32_t)k << kManyRowBits) + row;
    if (group == 0 && r < s.rows) {
#pragma unroll
      for (int i = 1; i < kJoinGroups; ++i) v.add(sums[i][row]);
      put_weight(p, b, r, old_weight(p, b, s, r), v.sum);
    }
    __syncthreads();
  }
}

template <int L, int NC>
void launch_few(const WeighParams& p, hipStream_t stream) {
  if (p.num_slots <= 1024) weigh_few_kernel<L, NC, 1024><<<kFewGrid, kFewBlock, 0, stream>>>(p);
  else weigh_few_kernel<L, NC, kMaxSlots + 1><<<kFewGrid, kFewBlock, 0, stream>>>(p);
}

template <int L>
void launch_weigh_as(const WeighParams& p, int64_t slot_queries, hipStream_t stream) {
  if (slot_queries <= 32) return launch_few<L, 1>(p, stream);
  if (slot_queries <= 64) return launch_few<L, 2>(p, stream);
  if (slot_queries <= kWeighFew) return launch_few<L, 4>(p, stream);
  if (p.num_slots <= 1024) {
    weigh_many_kernel<L, 1024><<<kWeighWorkgroups, kManyBlock, 0, stream>>>(p);
    weigh_join_kernel<1024><<<kWeighWorkgroups, kJoinBlock, 0, stream>>>(p);
  } else {
    weigh_many_kernel<L, kMaxSlots + 1><<<kWeighWorkgroups, kManyBlock, 0, stream>>>(p);
    weigh_join_kernel<kMaxSlots + 1><<<kWeighWorkgroups, kJoinBlock, 0, stream>>>(p);
  }
}

}  // namespace

hipError_t launch_weigh(const WeighParams& p, int64_t slot_queries, hipStream_t stream) {
  switch (p.cache.layout) {
    case kV4: launch_weigh_as<kV4>(p, slot_queries, stream); break;
    case kV41: launch_weigh_as<kV41>(p, slot_queries, stream); break;
    default: launch_weigh_as<kV41Fp4>(p, slot_queries, stream); break;
  }
  return hipGetLastError();
}

}  // namespace kvc
