// attend.hip -- attention over the paged compressed cache (gfx950): drafted
// tokens (a tree, a chain, one token) and packed causal prompts.
//
// A cached row x_r is key and value at once (512 dims, one row for all H query
// heads), so for a query q over its visible rows
//   s_r = scale * q . x_r,   out = sum_r e^(s_r) x_r / (sum_r e^(s_r) + e^sink)
// and one staged tile of rows serves both products.
//
// The queries of a slot are its (token, head) pairs in that order, cut into
// units of QT = 32 QB; a unit's rows are cut into tiles of NT = 128 / QB.
// Three launches: attend_plan_kernel deals the tiles of all units evenly to
// the workgroups of attend_kernel (one per compute unit, each a run of
// consecutive tiles, crossing units as it comes), and attend_join_kernel
// joins the units that were cut between workgroups.  The split follows the
// lengths on the device, so a captured call adapts to refreshed lengths, and
// it is a function of the lengths alone, so results repeat bit for bit.
#include "launch.hpp"
#include "row_load.hpp"

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

// ------------------------------------------------------------------ plan
// One workgroup: a prefix sum of the slots' units, then each thread walks an
// equal share of the units twice, to sum their tiles and to place the
// boundaries between the workgroups of attend_kernel.
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
  int64_t mine = 0, total = 0;
  walk([&](int, int32_t, int64_t t) { mine += t; });
  int64_t c = plan_excl_scan(mine, buf, &total);
  int64_t quota = (total + kAttendGrid - 1) / kAttendGrid;
  const int64_t least = kAttendLeastRows / nt;
  if (quota < least) quota = least;
  if (tid == 0) p.head->quota = quota;
  for (int64_t w = tid; w < kAttendGrid; w += kPlanBlock)
    if (w * quota >= total) p.starts[w].slot = -1;
  walk([&](int b, int32_t k, int64_t t) {
    const int64_t w0 = c / quota, w1 = (c + t - 1) / quota;
    for (int64_t w = w0 * quota == c ? w0 : w0 + 1; w <= w1; ++w)
      p.starts[w] = AttendStart{b, k, (int32_t)(w * quota - c), 0};
    if (w1 > w0)
      p.splits[atomicAdd(&nsplit, 1)] = AttendSplit{b, k, (int32_t)w0, (int32_t)(w1 - w0 + 1)};
    c += t;
  });
  __syncthreads();
  if (tid == 0) p.head->nsplit = nsplit;
}

// ------------------------------------------------------------------ attend
// The 16-byte chunks of an LDS row are permuted by the row index, so that a
// product's reads of one chunk column over many rows spread over the banks.
__device__ __forceinline__ uint32_t swz(uint32_t row) { return row & 7u; }

__device__ __forceinline__ float swap_halves(float v) { return __shfl_xor(v, 32); }

// Four steps of 16 dims of a 32 x 32 score block.  Written out so that the
// scores live in the vector registers their softmax works in: the compiler
// gives every matrix-instruction result of a kernel with an accumulator
// register file to that file, which O fills (256 registers for QB = 4).  A
// result feeding the next instruction's C operand needs no wait; s_nop 1
// covers operands a vector instruction has just written, and score_done's
// s_nop the 16 wait states from the last result to its first use.
__device__ __forceinline__ void score_mfma4(f32x16& sc, const bf16x8 (&x)[4], const bf16x8* q,
                                            bool first) {
  if (first)
    asm("s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %1, %5, 0\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %2, %6, %0\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %3, %7, %0\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %4, %8, %0"
        : "=&v"(sc)
        : "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3]));
  else
    asm("s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %1, %5, %0\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %2, %6, %0\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %3, %7, %0\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %4, %8, %0"
        : "+&v"(sc)
        : "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3]));
}
__device__ __forceinline__ void score_done(f32x16& sc) { asm("s_nop 15" : "+v"(sc)); }

// One step of 16 rows of O^T for a dim block and QB query blocks, O kept in
// accumulator registers; out_done stands before vector instructions read it.
template <int QB>
__device__ __forceinline__ void out_mfma(f32x16 (&o)[QB], bf16x8 x, const bf16x8 (&w)[QB]) {
  if constexpr (QB == 1)
    asm("s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0"
        : "+a"(o[0]) : "v"(x), "v"(w[0]));
  else if constexpr (QB == 2)
    asm("s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %2, %3, %0\n\t"
        "v_mfma_f32_32x32x16_bf16 %1, %2, %4, %1"
        : "+a"(o[0]), "+a"(o[1]) : "v"(x), "v"(w[0]), "v"(w[1]));
  else
    asm("s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %4, %5, %0\n\t"
        "v_mfma_f32_32x32x16_bf16 %1, %4, %6, %1\n\t"
        "v_mfma_f32_32x32x16_bf16 %2, %4, %7, %2\n\t"
        "v_mfma_f32_32x32x16_bf16 %3, %4, %8, %3"
        : "+a"(o[0]), "+a"(o[1]), "+a"(o[2]), "+a"(o[3])
        : "v"(x), "v"(w[0]), "v"(w[1]), "v"(w[2]), "v"(w[3]));
}
__device__ __forceinline__ void out_done(f32x16& o) { asm("s_nop 15" : "+a"(o)); }

// One workgroup, one unit's tiles at a time: scores S^T[row][query] = X Q^T
// with each wave on one 32 x 32 block (a lane owns one query, so the softmax
// statistics are per lane), the weights through LDS as bf16, then
// O^T[dim][query] += X^T P^T with each wave on 128 of the 512 dims.  X^T comes
// out of the same LDS tile by transposing reads.
//
// The weights are rounded to bf16 for the matrix product, the one rounding
// before the output's own; the sum they are divided by is of the rounded
// weights, so the division undoes a common part of it, while lse uses the
// exact weights.  The running maximum moves only when it is passed by 8 (in
// log2): weights up to 2^8 lose nothing in fp32, and O is rescaled rarely.
template <int L, int QB>
__global__ __launch_bounds__(kAttendBlock) __attribute__((amdgpu_waves_per_eu(1, 1)))
void attend_kernel(AttendParams p) {
  constexpr int NB = 4 / QB;
  constexpr int QT = 32 * QB, NT = 32 * NB;
  constexpr int RW = NT / 4;                  // rows a wave stages per tile
  constexpr int PS = NT + 8;                  // elements per query in the weights' tile
  __shared__ __attribute__((aligned(1024))) uint8_t tile[NT * 1024];
  __shared__ __attribute__((aligned(16))) uint16_t wts[QT * PS];
  __shared__ float smax[NB][QT], ssum[NB][QT], srsum[NB][QT], salpha[QT], sfac[QT];
  __shared__ __attribute__((aligned(16))) uint8_t svalid[16];
  __shared__ int32_t sscale[4], snf[4];
  const int lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  const int ql = lane & 31, h = lane >> 5;
  const int qb = wave % QB, nb = wave / QB;
  const PagedKV<L> kv{p.cache.base, p.cache.page_stride, p.cache.num_pages, p.cache.page_bits};
  const int32_t H = p.heads;
  const float c2 = p.scale_log2;

  // this lane's LDS addresses: row ql of the wave's score block, and the
  // transposing reads of its dim blocks
  // (the permutation touches the low 3 bits of a chunk's index only, so a few
  // bases and constant offsets reach every chunk)
  typedef const __attribute__((address_space(3))) uint8_t* lds_ptr;
  const lds_ptr tile3 = (lds_ptr)tile;
  const int i16 = lane & 15, g1 = (lane >> 4) & 1;
  lds_ptr kp[4], vp[2][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) kp[k] = tile3 + (nb * 32 + ql) * 1024 + (((2 * k + h) ^ swz(ql)) << 4);
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const int rr = 8 * h + 4 * e + (i16 >> 2);
      const int chunk = (4 * d + 2 * g1 + ((i16 >> 1) & 1)) ^ swz(rr);
      vp[e][d] = tile3 + rr * 1024 + 256 * wave + (chunk << 4) + 8 * (i16 & 1);
    }

  const AttendStart st = p.starts[blockIdx.x];
  int b = st.slot, ub = st.unit;
  int32_t t0 = st.tile;
  int64_t left = p.head->quota;
  int32_t none = 0;
  bool first_piece = true;
  if (b < 0) return;
  SlotTokens s = slot_tokens(p, b, &none);

  while (left > 0) {
    // ---- the piece: tiles [t0, t1) of unit ub of slot b
    const int32_t nq = s.n * H, m0 = ub * QT;
    const int32_t rows = unit_rows(p, s, m0, QT);
    const int32_t tiles = unit_tiles(rows, NT);
    const int32_t t1 = (int32_t)min((int64_t)tiles, t0 + left);
    const int32_t* pt = p.page_table + (int64_t)b * p.pt_stride;

    // this lane's query
    // (one past the slot's last takes the last one's place; nothing of it is
    // written)
    const bool qok = m0 + qb * 32 + ql < nq;
    const int32_t m = qok ? m0 + qb * 32 + ql : nq - 1;
    const int32_t tok = (int32_t)udiv_magic((uint32_t)m, p.head_div.m, p.head_div.sh1,
                                            p.head_div.sh2);
    const int32_t head = m - tok * H;
    const uint16_t* qp = p.q + (int64_t)(s.first + tok) * p.q_stride + (int64_t)head * p.q_hstride;
    bf16x8 q[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      q[k] = __builtin_bit_cast(bf16x8, ld_u4(qp + 16 * k + 8 * h));
    }
    // rows below lim are visible; of the rows from base on, those of bits
    int32_t lim;
    uint64_t bits = 0;
    const int32_t base = s.pos;
    int32_t lim_first;                        // every query sees the rows below
    if (p.tree != nullptr) {
      lim = s.pos;
      bits = p.tree[(int64_t)b * p.draft_len + tok];
      if (s.n < 64) bits &= (uint64_t(1) << s.n) - 1;
      lim_first = s.pos;
    } else {
      lim = (s.pos + tok + 1) >> (p.ratio - 1);
      const int32_t tok0 = (int32_t)udiv_magic((uint32_t)m0, p.head_div.m, p.head_div.sh1,
                                               p.head_div.sh2);
      lim_first = (s.pos + tok0 + 1) >> (p.ratio - 1);
    }

    // row r's page-table entry, row r's slot
    auto page_of = [&](int32_t tl) -> int32_t {
      const int32_t r = tl * NT + wave * RW + lane;
      const int32_t lp = r >> p.cache.page_bits;
      if (lane >= RW || tl >= t1 || r >= rows) return -1;
      if (lp >= p.pt_width) {
        if (p.status != nullptr) atomicOr(p.status, kStPtRange);
        return -1;
      }
      return pt[lp];
    };
    auto slot_of = [&](int32_t tl, int32_t page) -> int32_t {
      const int32_t r = tl * NT + wave * RW + lane;
      if (lane >= RW || tl >= t1 || r >= rows || (r >> p.cache.page_bits) >= p.pt_width) return -1;
      if (page < 0 || page >= kv.num_pages) {
        if (p.status != nullptr) atomicOr(p.status, kStPageRange);
        return -1;
      }
      return (page << p.cache.page_bits) | (r & ((1 << p.cache.page_bits) - 1));
    };
    LaneCodes<L> codes[RW];
    int32_t slot = slot_of(t0, page_of(t0));
    // a row without a slot loads slot 0 (any cache has one) and is zeroed below
#pragma unroll
    for (int u = 0; u < RW; ++u) {
      const int32_t sl = __builtin_amdgcn_readlane(slot, u);
      codes[u] = load_lane<L, kCpolSc1>(kv, sl < 0 ? 0 : sl, lane);
    }
    int32_t page = page_of(t0 + 1);

    float mx = kNegInf, sum = 0.0f, rsum = 0.0f;
    f32x16 o[4][QB];
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int x = 0; x < QB; ++x) o[d][x] = f32x16{};

    for (int32_t tl = t0; tl < t1; ++tl) {
      // ---- stage the tile's rows, request the next tile's
      const uint64_t okm = __ballot(slot >= 0);
#pragma unroll
      for (int u = 0; u < RW; ++u) {
        const int row = wave * RW + u;
        uint4 v = decode_lane<L>(codes[u], lane);
        if ((okm >> u & 1) == 0) v = make_uint4(0, 0, 0, 0);
        *(u32x4*)(tile + row * 1024 + ((lane ^ swz(row)) << 4)) = u32x4{v.x, v.y, v.z, v.w};
      }
      if (lane < RW / 8) svalid[wave * (RW / 8) + lane] = (uint8_t)(okm >> (8 * lane));
      if (tl + 1 < t1) {
        slot = slot_of(tl + 1, page);
#pragma unroll
        for (int u = 0; u < RW; ++u) {
          const int32_t sl = __builtin_amdgcn_readlane(slot, u);
          codes[u] = load_lane<L, kCpolSc1>(kv, sl < 0 ? 0 : sl, lane);
        }
        page = page_of(tl + 2);
      }
      __syncthreads();

      // ---- scores of this wave's 32 rows and 32 queries
      f32x16 sc;
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        bf16x8 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = __builtin_bit_cast(
              bf16x8, *(const __attribute__((address_space(3))) u32x4*)(kp[i] + 32 * k));
        score_mfma4(sc, x, q + k, k == 0);
      }
      score_done(sc);
      // ---- mask (only a tile that some query does not see whole)
      bool holes = (tl + 1) * NT > lim_first;
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) holes |= *(const uint32_t*)(svalid + 4 * w) != 0xFFFFFFFFu;
      if (holes) {
        const uint32_t okw = *(const uint32_t*)(svalid + 4 * nb);
        bool nf = false;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int rl = 8 * (i >> 2) + 4 * h + (i & 3);
          const int32_t r = tl * NT + nb * 32 + rl;
          bool see = r < lim;
          if (p.tree != nullptr) {
            const uint32_t x = (uint32_t)(r - base);
            see |= x < 64u && (bits >> x & 1) != 0;
          }
          see &= (okw >> rl & 1) != 0;
          nf |= !see && !(__builtin_fabsf(sc[i]) < __builtin_inff());
          sc[i] = see ? sc[i] : kNegInf;
        }
        const bool any = __ballot(nf) != 0;
        if (lane == 0) snf[wave] = any;
      }
      // ---- the query's new reference maximum
      float tm = sc[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) tm = fmaxf(tm, sc[i]);
      tm = fmaxf(tm, swap_halves(tm));
      if constexpr (NB > 1) {
        if (h == 0) smax[nb][qb * 32 + ql] = tm;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < NB; ++x) tm = fmaxf(tm, smax[x][qb * 32 + ql]);
      }
      tm *= c2;
      const float old = mx;
      if (tm > mx + 8.0f) mx = tm;
      const float alpha = mx == old ? 1.0f : __builtin_amdgcn_exp2f(old - mx);
      const float ref = mx == kNegInf ? 0.0f : mx;
      sum *= alpha;
      rsum *= alpha;
      // ---- weights, their sums, and their bf16 to LDS
      uint16_t* const wrow = wts + (qb * 32 + ql) * PS + nb * 32 + 4 * h;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[4 * j + i], c2, -ref));
          sum += e[i];
        }
        const uint32_t w0 = pack_bf16(e[0], e[1]), w1 = pack_bf16(e[2], e[3]);
        rsum += (bf16_lo(w0) + bf16_hi(w0)) + (bf16_lo(w1) + bf16_hi(w1));
        *(u32x2*)(wrow + 8 * j) = u32x2{w0, w1};
      }
      const bool rescale = __ballot(alpha != 1.0f) != 0;
      if (nb == 0) {
        if (h == 0) salpha[qb * 32 + ql] = alpha;
        if (lane == 0) sscale[qb] = rescale;
      }
      __syncthreads();
      // ---- a NaN or an infinity in a row that some query does not see: its
      // weight there is 0, and 0 times it would not be
      if (holes) {
        int32_t any = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) any |= snf[w];
        if (any != 0) {
          for (int x = threadIdx.x; x < NT * 64; x += kAttendBlock) {
            u32x4 v = *(u32x4*)(tile + 16 * x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if ((v[k] & 0x7F80u) == 0x7F80u) v[k] &= 0xFFFF0000u;
              if ((v[k] & 0x7F800000u) == 0x7F800000u) v[k] &= 0xFFFFu;
            }
            *(u32x4*)(tile + 16 * x) = v;
          }
          __syncthreads();
        }
      }
      // ---- O += X^T P^T on dims [128 wave, 128 wave + 128)
#pragma unroll
      for (int x = 0; x < QB; ++x) {
        if (sscale[x] == 0) continue;
        const float a = salpha[x * 32 + ql];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          out_done(o[d][x]);
          o[d][x] *= a;
        }
      }
#pragma unroll
      for (int k = 0; k < NT / 16; ++k) {
        bf16x8 w[QB];
#pragma unroll
        for (int x = 0; x < QB; ++x)
          w[x] = __builtin_bit_cast(bf16x8, *(const u32x4*)(wts + (x * 32 + ql) * PS + 16 * k + 8 * h));
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          union { s16x4 half[2]; bf16x8 v; } x;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            x.half[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(vp[e][d & 1] + 128 * (d >> 1) +
                                                           16384 * k));
          out_mfma<QB>(o[d], x.v, w);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();                        // the tile and the weights are free
    }

#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int x = 0; x < QB; ++x) out_done(o[d][x]);
    // ---- the piece's end: its sums over the lanes and waves of a query
    sum += swap_halves(sum);
    rsum += swap_halves(rsum);
    const int qi = qb * 32 + ql;
    if (h == 0) { ssum[nb][qi] = sum; srsum[nb][qi] = rsum; }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == tiles;
    const int64_t part = ((int64_t)blockIdx.x * 2 + (first_piece && t0 > 0 ? 0 : 1));
    if (nb == 0) {
      sum = ssum[0][qi];
      rsum = srsum[0][qi];
#pragma unroll
      for (int x = 1; x < NB; ++x) { sum += ssum[x][qi]; rsum += srsum[x][qi]; }
      if (whole) {
        const float snk = p.sink != nullptr ? p.sink[head] * kLog2e : kNegInf;
        const float mm = fmaxf(mx, snk);
        const float e = mx == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mx - mm);
        const float es = snk == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(snk - mm);
        if (h == 0) {
          sfac[qi] = e == 0.0f ? 0.0f : e / (rsum * e + es);
          if (p.lse != nullptr && qok)
            p.lse[(int64_t)(s.first + tok) * H + head] = mm + __builtin_log2f(sum * e + es);
        }
      } else if (h == 0) {
        p.part_ml[part * QT + qi] = make_float4(mx, sum, rsum, 0.0f);
      }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < QB; ++x) {
      const int32_t mq = m0 + x * 32 + ql;
      if (mq < nq) {
        const int32_t tk = (int32_t)udiv_magic((uint32_t)mq, p.head_div.m, p.head_div.sh1, p.head_div.sh2);
        uint16_t* op = p.out + (int64_t)(s.first + tk) * p.out_stride + (int64_t)(mq - tk * H) * p.out_hstride;
        float* pp = p.part_o + (part * QT + x * 32 + ql) * kDim;
        const float f = whole ? sfac[x * 32 + ql] : 1.0f;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int dim = 128 * wave + 32 * d + 8 * j + 4 * h;
            const float a0 = o[d][x][4 * j], a1 = o[d][x][4 * j + 1], a2 = o[d][x][4 * j + 2],
                        a3 = o[d][x][4 * j + 3];
            if (whole)
              *(u32x2*)(op + dim) = u32x2{pack_bf16(a0 * f, a1 * f), pack_bf16(a2 * f, a3 * f)};
            else
              *(f32x4*)(pp + dim) = f32x4{a0, a1, a2, a3};
          }
        }
      }
    }
    __syncthreads();

    // ---- the next piece
    left -= t1 - t0;
    t0 = 0;
    first_piece = false;
    ++ub;
    if (left > 0 && (int64_t)ub * QT >= (int64_t)s.n * H) {
      ub = 0;
      // the next slot that has tokens, 64 at a time
      int bn = b + 1;
      for (;;) {
        if (bn >= p.num_slots) return;
        SlotTokens c{};
        if (bn + lane < p.num_slots) c = slot_tokens(p, bn + lane, &none);
        const uint64_t has = __ballot(c.n > 0);
        if (has != 0) {
          b = bn + __builtin_ctzll(has);
          break;
        }
        bn += kLanes;
      }
      s = slot_tokens(p, b, &none);
    }
  }
}

// ------------------------------------------------------------------ join
// One workgroup per query of a unit that was cut: the parts are dealt to the
// four waves (8 dims a lane), each scaled to the common maximum, and the
// waves' sums added.
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p, int qt) {
  __shared__ float acc[3][kDim];
  if ((int)blockIdx.x >= p.head->nsplit) return;
  const AttendSplit sp = p.splits[blockIdx.x];
  int32_t none = 0;
  const SlotTokens s = slot_tokens(p, sp.slot, &none);
  const int qi = blockIdx.y;
  const int32_t m = sp.unit * qt + qi;
  if (m >= s.n * p.heads) return;
  const int lane = lane_id(), wave = uniform((int)(threadIdx.x >> 6));
  // part k lies with workgroup wg0 + k: its second place for the first part
  // (which began at the unit's first tile), its first place for the others
  auto place = [&](int k) -> int64_t { return ((int64_t)(sp.wg0 + k) * 2 + (k == 0 ? 1 : 0)) * qt + qi; };
  float mx = kNegInf;
  for (int k = lane; k < sp.parts; k += kLanes) mx = fmaxf(mx, p.part_ml[place(k)].x);
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  float sum = 0.0f, rsum = 0.0f;
  for (int k = lane; k < sp.parts; k += kLanes) {
    const float4 v = p.part_ml[place(k)];
    const float e = v.x == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(v.x - mx);
    sum += v.y * e;
    rsum += v.z * e;
  }
  sum = wave_sum_f32(sum);
  rsum = wave_sum_f32(rsum);
  float a[8] = {};
  for (int k = wave; k < sp.parts; k += 4) {
    const int64_t at = place(k);
    const float4 v = p.part_ml[at];
    if (v.y == 0.0f) continue;                // a part that saw nothing
    const float e = v.x == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(v.x - mx);
    const f32x4 x = *(const f32x4*)(p.part_o + at * kDim + 8 * lane);
    const f32x4 y = *(const f32x4*)(p.part_o + at * kDim + 8 * lane + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = __builtin_fmaf(x[i], e, a[i]);
      a[4 + i] = __builtin_fmaf(y[i], e, a[4 + i]);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[wave - 1][8 * lane + i] = a[i];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] += acc[w][8 * lane + i];
  const int32_t tok = (int32_t)udiv_magic((uint32_t)m, p.head_div.m, p.head_div.sh1, p.head_div.sh2);
  const int32_t head = m - tok * p.heads;
  const float snk = p.sink != nullptr ? p.sink[head] * kLog2e : kNegInf;
  const float mm = fmaxf(mx, snk);
  const float e = mx == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mx - mm);
  const float es = snk == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(snk - mm);
  const float f = e == 0.0f ? 0.0f : e / (rsum * e + es);
  uint16_t* op = p.out + (int64_t)(s.first + tok) * p.out_stride + (int64_t)head * p.out_hstride;
  st_u4(op + 8 * lane, make_uint4(pack_bf16(a[0] * f, a[1] * f), pack_bf16(a[2] * f, a[3] * f),
                                  pack_bf16(a[4] * f, a[5] * f), pack_bf16(a[6] * f, a[7] * f)));
  if (p.lse != nullptr && lane == 0)
    p.lse[(int64_t)(s.first + tok) * p.heads + head] = mm + __builtin_log2f(sum * e + es);
}

template <int L>
hipError_t attend(const AttendParams& p, int qblocks, hipStream_t stream) {
  const dim3 grid(kAttendGrid), block(kAttendBlock);
  switch (qblocks) {
    case 1: hipLaunchKernelGGL((attend_kernel<L, 1>), grid, block, 0, stream, p); break;
    case 2: hipLaunchKernelGGL((attend_kernel<L, 2>), grid, block, 0, stream, p); break;
    default: hipLaunchKernelGGL((attend_kernel<L, 4>), grid, block, 0, stream, p); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attend(const AttendParams& p, int qblocks, hipStream_t stream) {
  const int qt = 32 * qblocks, nt = 128 / qblocks;
  hipLaunchKernelGGL(attend_plan_kernel, dim3(1), dim3(kPlanBlock), 0, stream, p, qt, nt);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  switch (p.cache.layout) {
    case kV41: e = attend<kV41>(p, qblocks, stream); break;
    case kV41Fp4: e = attend<kV41Fp4>(p, qblocks, stream); break;
    default: e = attend<kV4>(p, qblocks, stream); break;
  }
  if (e != hipSuccess) return e;
  // a unit cut between workgroups holds at least one boundary between two
  const int64_t splits = p.units_max < kAttendGrid - 1 ? p.units_max : kAttendGrid - 1;
  hipLaunchKernelGGL(attend_join_kernel, dim3((unsigned)splits, (unsigned)qt), dim3(256), 0, stream,
                     p, qt);
  return hipGetLastError();
}

}  // namespace kvc
