// kvc_api.cpp -- the C ABI (include/kvc.h): argument checks from host
// scalars, dispatch to the kernel launchers, error strings and the host-side
// dequant-reuse head.  Nothing here touches device memory or synchronises.
#include "../../include/kvc.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>
#include <cstring>
#include <string>

#include "launch_evict.hpp"

namespace {

thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int ok() {
  g_last_error.clear();
  return KVC_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool layout_info(int32_t layout, kvc_layout_info* info) {
  switch (layout) {
    case KVC_LAYOUT_V4: *info = {576, 8, 584, 64, 448}; return true;
    case KVC_LAYOUT_V41: *info = {512, 16, 528, 32, 512}; return true;
    case KVC_LAYOUT_V41_FP4: *info = {256, 32, 288, 16, 512}; return true;
    default: return false;
  }
}

int page_bits_of(int32_t page_size) {
  int b = 0;
  while ((1 << b) < page_size) ++b;
  return b;
}

// checks the cache descriptor and fills the device view
int check_cache(const kvc_cache* c, kvc::CacheView* v, const char* who) {
  if (c == nullptr) return fail(KVC_EINVAL, "%s: cache descriptor is NULL", who);
  kvc_layout_info li;
  if (!layout_info(c->layout, &li)) return fail(KVC_EUNSUPPORTED, "%s: unknown layout %d", who, c->layout);
  if (c->base == nullptr) return fail(KVC_EINVAL, "%s: cache base is NULL", who);
  if (!aligned16(c->base)) return fail(KVC_EINVAL, "%s: cache base is not 16-byte aligned", who);
  if (c->page_size < 1 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0)
    return fail(KVC_EINVAL, "%s: page_size %d is not a power of two in [1, 4096]", who, c->page_size);
  if (c->page_stride < (int64_t)c->page_size * li.row_bytes || c->page_stride % 16 != 0)
    return fail(KVC_EINVAL, "%s: page_stride %lld must be >= page_size * %d and a multiple of 16",
                who, (long long)c->page_stride, li.row_bytes);
  if (c->num_pages < 1) return fail(KVC_EINVAL, "%s: num_pages must be >= 1", who);
  if (c->num_pages > ((int64_t)1 << 31) / c->page_size)
    return fail(KVC_EINVAL, "%s: num_pages * page_size must fit in int32 slots", who);
  v->base = static_cast<uint8_t*>(c->base);
  v->page_stride = c->page_stride;
  v->num_pages = c->num_pages;
  v->page_bits = page_bits_of(c->page_size);
  v->layout = c->layout;
  return KVC_OK;
}

bool row_stride_ok(int64_t s) { return s >= 512 && s % 8 == 0; }

int launched(hipError_t e, const char* who) {
  if (e != hipSuccess) return fail(KVC_ELAUNCH, "%s: launch failed: %s", who, hipGetErrorString(e));
  return ok();
}

bool page_size_ok(int32_t ps) { return ps >= 1 && ps <= 4096 && (ps & (ps - 1)) == 0; }

// 32-query blocks per unit of the attention.  A unit's wider tiles cost fewer
// reads of the staged rows per query, a wide unit half full costs its empty
// half: slots of up to 32 or 64 queries take units of that size.  Measured, a
// token of 64 requests over V41_FP4 rows: 64 heads 123 us in units of 64, 172 in
// units of 128; 32 heads 104 us in units of 32, 124 in units of 64.  The rule sees
// the call's sizes, not the lengths, which are on the device: a packed step of a
// 2,048-token prompt and 200 single tokens with 16 heads averages 180 queries a
// slot and takes units of 128, 304 us where the prompt alone takes 114 and the
// tokens alone 131.
int attend_qblocks(int32_t slots, int64_t tokens, int32_t heads) {
  const int64_t per_slot = tokens * heads / (slots > 0 ? slots : 1);
  return per_slot <= 32 ? 1 : per_slot <= 64 ? 2 : 4;
}

constexpr int64_t kMaxQueries = 0x7FFFFF00;   // query indices, rounded up to a unit, stay in int32

int64_t align256(int64_t n) { return (n + 255) & ~int64_t(255); }

// places of the workspace's parts; returns where they end
int64_t attend_layout(int32_t slots, int64_t tokens, int32_t heads, int64_t (&at)[5]) {
  const int64_t parts = 2 * int64_t(kvc::kAttendWorkgroups) * 32 * attend_qblocks(slots, tokens, heads);
  int64_t n = 0;
  at[0] = n, n += align256(sizeof(kvc::AttendHead));
  at[1] = n, n += align256((kvc::kAttendWorkgroups + 1) * sizeof(kvc::AttendStart));
  at[2] = n, n += align256(kvc::kAttendPlanUnits * sizeof(kvc::AttendSplit));
  at[3] = n, n += align256(parts * 16);
  at[4] = n, n += align256(parts * 512 * 4);
  return n;
}

// bytes for `tokens` token rows whatever slots they are in: those of the widest
// units they may take, one slot's (so that a workspace for the largest batch
// serves the smaller ones, whose units may be wider)
int64_t attend_bytes(int64_t tokens, int32_t heads) {
  int64_t at[5];
  return attend_layout(1, tokens, heads, at);
}

// the checks and the call shared by both attention entry points
int attend(const kvc_attend_args* a, bool tree, void* stream, const char* who) {
  if (a == nullptr) return fail(KVC_EINVAL, "%s: args is NULL", who);
  kvc::AttendParams p{};
  int rc = check_cache(&a->cache, &p.cache, who);
  if (rc) return rc;
  if (a->ratio != 1 && a->ratio != 2) return fail(KVC_EUNSUPPORTED, "%s: ratio %d (1 or 2)", who, a->ratio);
  if (a->num_heads < 1 || a->num_heads > 1024)
    return fail(KVC_EINVAL, "%s: num_heads %d outside [1, 1024]", who, a->num_heads);
  if (a->num_slots < 0 || a->num_slots > kvc::kMaxSlots)
    return fail(KVC_EINVAL, "%s: num_slots %d outside [0, %d]", who, a->num_slots, kvc::kMaxSlots);
  if (a->q_rows < 0 || a->q_rows > kMaxQueries / a->num_heads)
    return fail(KVC_EINVAL, "%s: q_rows %lld: q_rows * num_heads must not pass 2^31 - 256", who,
                (long long)a->q_rows);
  if (tree) {
    if (a->draft_len < 1 || a->draft_len > 64)
      return fail(KVC_EINVAL, "%s: draft_len %d outside [1, 64]", who, a->draft_len);
    if (a->tree != nullptr && a->ratio != 1)
      return fail(KVC_EUNSUPPORTED, "%s: a tree needs ratio 1 (a cached row per drafted token)", who);
    if (a->q_rows < (int64_t)a->num_slots * a->draft_len)
      return fail(KVC_EINVAL, "%s: q_rows %lld, need num_slots * draft_len = %lld", who,
                  (long long)a->q_rows, (long long)a->num_slots * a->draft_len);
  }
  if (a->num_slots == 0 || a->q_rows == 0) return ok();
  if (a->q == nullptr || !aligned16(a->q) || a->out == nullptr || !aligned16(a->out))
    return fail(KVC_EINVAL, "%s: q and out must be non-NULL and 16-byte aligned", who);
  // (the stride of an axis of one entry is not used)
  p.q_stride = a->q_rows > 1 ? a->q_stride : 0;
  p.q_hstride = a->num_heads > 1 ? a->q_head_stride : 0;
  p.out_stride = a->q_rows > 1 ? a->out_stride : 512;
  p.out_hstride = a->num_heads > 1 ? a->out_head_stride : 512;
  if (p.q_stride < 0 || p.q_hstride < 0 || p.q_stride % 8 != 0 || p.q_hstride % 8 != 0)
    return fail(KVC_EINVAL, "%s: q strides must be multiples of 8, >= 0", who);
  if (p.out_stride % 8 != 0 || p.out_hstride % 8 != 0 || p.out_stride < 512 || p.out_hstride < 512)
    return fail(KVC_EINVAL, "%s: out strides must be multiples of 8, >= 512", who);
  if (a->start_pos == nullptr) return fail(KVC_EINVAL, "%s: start_pos is NULL", who);
  if (!tree && a->offsets == nullptr) return fail(KVC_EINVAL, "%s: offsets is NULL", who);
  if (a->page_table == nullptr || a->pt_width < 1 || a->pt_stride < a->pt_width)
    return fail(KVC_EINVAL, "%s: page table needs 1 <= pt_width <= pt_stride (%lld, %lld)", who,
                (long long)a->pt_width, (long long)a->pt_stride);
  p.scale_log2 = (float)((double)a->scale * 1.4426950408889634074);
  if (!(a->scale > 0.0f) || !std::isfinite(p.scale_log2))
    return fail(KVC_EINVAL, "%s: scale must be > 0, and scale * log2(e) finite", who);
  const int64_t tokens = tree ? (int64_t)a->num_slots * a->draft_len : a->q_rows;
  const int64_t need = attend_bytes(tokens, a->num_heads);
  if (a->workspace == nullptr || ((uintptr_t)a->workspace & 255u) != 0 || a->workspace_bytes < need)
    return fail(KVC_EINVAL, "%s: workspace needs %lld bytes, 256-byte aligned", who, (long long)need);
  if (kvc::launch_attend == nullptr) return fail(KVC_ELAUNCH, "%s: built without kernels", who);
  p.ratio = a->ratio;
  p.heads = a->num_heads;
  p.head_div = kvc::div_magic((uint32_t)a->num_heads);
  p.num_slots = a->num_slots;
  p.draft_len = tree ? a->draft_len : 0;
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_rows = a->q_rows;
  p.offsets = tree ? nullptr : a->offsets;
  p.start_pos = a->start_pos;
  p.page_table = a->page_table;
  p.pt_stride = a->pt_stride;
  p.pt_width = a->pt_width;
  p.tree = tree ? a->tree : nullptr;
  p.sink = a->sink;
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.status = a->status;
  int qblocks = attend_qblocks(a->num_slots, tokens, a->num_heads);
  if (a->cache.page_size < 8 && qblocks == 4) qblocks = 2;   // the wide kernel's pages hold 8 rows or more
  p.units_max = tokens * a->num_heads / (32 * qblocks) + a->num_slots;
  const int64_t units =
      ((tree ? a->draft_len : tokens) * a->num_heads + 32 * qblocks - 1) / (32 * qblocks);
  if (units * a->num_slots <= kvc::kAttendPlanUnits) {
    p.plan_units = (int32_t)units;
    p.plan_div = kvc::div_magic((uint32_t)units);
  }
  int64_t at[5];
  attend_layout(a->num_slots, tokens, a->num_heads, at);
  uint8_t* w = static_cast<uint8_t*>(a->workspace);
  p.head = reinterpret_cast<kvc::AttendHead*>(w + at[0]);
  p.starts = reinterpret_cast<kvc::AttendStart*>(w + at[1]);
  p.splits = reinterpret_cast<kvc::AttendSplit*>(w + at[2]);
  p.part_ml = reinterpret_cast<float4*>(w + at[3]);
  p.part_o = reinterpret_cast<float*>(w + at[4]);
  return launched(kvc::launch_attend(p, qblocks, static_cast<hipStream_t>(stream)), who);
}

// ------------------------------------------------------------------ rotary
// pair index that makes `turns` turns over the original context
double pair_of_turns(const kvc_rope_table_args* a, double turns) {
  return a->rot_dim * std::log(a->original / (turns * 6.283185307179586477)) / (2.0 * std::log(a->base));
}

// speeds as half turns a position
void rope_speeds(const kvc_rope_table_args* a, double* speed) {
  const int R = a->rot_dim;
  const double base = a->scaling == KVC_ROPE_BASE ? a->base * std::pow(a->factor, double(R) / (R - 2)) : a->base;
  double lo = 0.0, hi = 0.0;
  if (a->scaling == KVC_ROPE_PARTS) {
    lo = std::fmax(std::floor(pair_of_turns(a, a->beta_fast)), 0.0);
    hi = std::fmin(std::ceil(pair_of_turns(a, a->beta_slow)), double(R - 1));
  }
  for (int j = 0; j < R / 2; ++j) {
    double w = std::pow(base, -2.0 * j / R);
    if (a->scaling == KVC_ROPE_LINEAR) {
      w /= a->factor;
    } else if (a->scaling == KVC_ROPE_PARTS) {
      const double r = std::fmin(std::fmax((j - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      w = w * (1.0 - r) + w / a->factor * r;
    }
    speed[j] = w / 3.141592653589793238;
  }
}

bool positive(double v) { return v > 0.0 && std::isfinite(v); }

// ------------------------------------------------------------------ weights
constexpr int64_t kWeighBytes =
    (int64_t)sizeof(kvc::WeighHead) + kvc::kWeighParts * kvc::kWeighRows * (int64_t)sizeof(float);

int weigh(const kvc_weigh_args* a, bool tree, void* stream, const char* who) {
  if (a == nullptr) return fail(KVC_EINVAL, "%s: args is NULL", who);
  kvc::WeighParams p{};
  int rc = check_cache(&a->cache, &p.cache, who);
  if (rc) return rc;
  if (a->ratio != 1 && a->ratio != 2) return fail(KVC_EUNSUPPORTED, "%s: ratio %d (1 or 2)", who, a->ratio);
  if (a->num_heads < 1 || a->num_heads > 1024)
    return fail(KVC_EINVAL, "%s: num_heads %d outside [1, 1024]", who, a->num_heads);
  if (a->num_slots < 0 || a->num_slots > kvc::kMaxSlots)
    return fail(KVC_EINVAL, "%s: num_slots %d outside [0, %d]", who, a->num_slots, kvc::kMaxSlots);
  if (a->q_rows < 0 || a->q_rows > kMaxQueries / a->num_heads)
    return fail(KVC_EINVAL, "%s: q_rows %lld: q_rows * num_heads must not pass 2^31 - 256", who,
                (long long)a->q_rows);
  if (tree) {
    if (a->draft_len < 1 || a->draft_len > 64)
      return fail(KVC_EINVAL, "%s: draft_len %d outside [1, 64]", who, a->draft_len);
    if (a->tree != nullptr && a->ratio != 1)
      return fail(KVC_EUNSUPPORTED, "%s: a tree needs ratio 1 (a cached row per drafted token)", who);
    if (a->q_rows < (int64_t)a->num_slots * a->draft_len)
      return fail(KVC_EINVAL, "%s: q_rows %lld, need num_slots * draft_len = %lld", who,
                  (long long)a->q_rows, (long long)a->num_slots * a->draft_len);
  }
  if (!(a->decay >= 0.0f) || !std::isfinite(a->decay))
    return fail(KVC_EINVAL, "%s: decay must be finite, >= 0", who);
  p.scale_log2 = (float)((double)a->scale * 1.4426950408889634074);
  if (!(a->scale > 0.0f) || !std::isfinite(p.scale_log2))
    return fail(KVC_EINVAL, "%s: scale must be > 0, and scale * log2(e) finite", who);
  if (a->num_slots == 0 || a->q_rows == 0) return ok();
  if (a->q == nullptr || !aligned16(a->q)) return fail(KVC_EINVAL, "%s: q must be non-NULL and 16-byte aligned", who);
  // (the stride of an axis of one entry is not used)
  p.q_stride = a->q_rows > 1 ? a->q_stride : 0;
  p.q_hstride = a->num_heads > 1 ? a->q_head_stride : 0;
  if (p.q_stride < 0 || p.q_hstride < 0 || p.q_stride % 8 != 0 || p.q_hstride % 8 != 0 ||
      p.q_stride > 0x7FFFFFFF || p.q_hstride > 0x7FFFFFFF)
    return fail(KVC_EINVAL, "%s: q strides must be multiples of 8 in [0, 2^31)", who);
  if (a->lse == nullptr || a->start_pos == nullptr || (!tree && a->offsets == nullptr))
    return fail(KVC_EINVAL, "%s: NULL lse, start_pos or offsets", who);
  if (a->page_table == nullptr || a->pt_width < 1 || a->pt_stride < a->pt_width)
    return fail(KVC_EINVAL, "%s: page table needs 1 <= pt_width <= pt_stride (%lld, %lld)", who,
                (long long)a->pt_width, (long long)a->pt_stride);
  if (a->weights == nullptr || a->w_width < 1 || a->w_stride < a->w_width)
    return fail(KVC_EINVAL, "%s: weights need 1 <= w_width <= w_stride (%lld, %lld)", who,
                (long long)a->w_width, (long long)a->w_stride);
  if (a->prev != nullptr && a->prev_stride < a->w_width)
    return fail(KVC_EINVAL, "%s: prev_stride %lld below w_width %lld", who, (long long)a->prev_stride,
                (long long)a->w_width);
  // (one slot's row has no next one)
  if (a->prev == a->weights && a->num_slots > 1 && a->prev_stride != a->w_stride)
    return fail(KVC_EINVAL, "%s: prev is weights, with another stride", who);
  if (a->weights == a->lse) return fail(KVC_EINVAL, "%s: weights must not be an input", who);
  const int64_t slot_queries = (tree ? (int64_t)a->draft_len : a->q_rows) * a->num_heads;
  if (slot_queries > kvc::kWeighFew &&
      (a->workspace == nullptr || ((uintptr_t)a->workspace & 255u) != 0 || a->workspace_bytes < kWeighBytes))
    return fail(KVC_EINVAL, "%s: workspace needs %lld bytes, 256-byte aligned", who, (long long)kWeighBytes);
  if (kvc::launch_weigh == nullptr) return fail(KVC_ELAUNCH, "%s: built without kernels", who);
  p.ratio = a->ratio;
  p.heads = a->num_heads;
  p.head_div = kvc::div_magic((uint32_t)a->num_heads);
  p.num_slots = a->num_slots;
  p.draft_len = tree ? a->draft_len : 0;
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_rows = a->q_rows;
  p.lse = a->lse;
  p.offsets = tree ? nullptr : a->offsets;
  p.start_pos = a->start_pos;
  p.page_table = a->page_table;
  p.pt_stride = a->pt_stride;
  p.pt_width = a->pt_width < 0x7FFFFFFF ? a->pt_width : 0x7FFFFFFF;   // (no row has a later page)
  p.tree = tree ? a->tree : nullptr;
  p.decay = a->decay;
  p.prev = a->decay == 0.0f ? nullptr : a->prev;   // (not read: 0 times anything)
  p.prev_stride = a->prev_stride;
  p.weights = a->weights;
  p.w_stride = a->w_stride;
  p.w_width = a->w_width;
  p.status = a->status;
  if (slot_queries > kvc::kWeighFew) {
    p.head = static_cast<kvc::WeighHead*>(a->workspace);
    p.parts = reinterpret_cast<float*>(p.head + 1);
  }
  return launched(kvc::launch_weigh(p, slot_queries, static_cast<hipStream_t>(stream)), who);
}

// ------------------------------------------------------------------ eviction
// segments of a slot's row of weights, 0 where it is not cut
int32_t evict_segments(int32_t slots, int64_t width) {
  if (width <= kvc::kSelectRegisterRows || slots < 1 || slots > kvc::kSelectSegmentSlots) return 0;
  const int64_t most = kvc::kSelectSegments / slots;
  const int64_t n = (width - 1) / kvc::kSelectSegmentRows + 1;
  return (int32_t)(n < most ? n : most);
}

// Bytes for calls of up to that many slots and weights a row, whatever cut
// they take: a shorter row, or fewer slots, may be cut into more segments in
// all, up to the most there are.
int64_t evict_bytes(int32_t slots, int64_t width) {
  if (width <= kvc::kSelectRegisterRows) return 0;
  const int64_t each = (width - 1) / kvc::kSelectSegmentRows + 1;
  const int64_t n = (each < kvc::kSelectSegments ? each : kvc::kSelectSegments) * slots;
  const int64_t segments = n < kvc::kSelectSegments ? n : kvc::kSelectSegments;
  return segments * (3 * kvc::kSelectWords + 4) * 4;
}

}  // namespace

// --------------------------------------------------------------------------
struct kvc_kvbuf {
  bool valid;
  void* base;
  int32_t layout;
  int32_t page_size;
  int64_t page_stride;
  const int32_t* page_table;
  int64_t n_pages;
  const int32_t* ids;
  int64_t n;
  void* out;
  int64_t out_stride;
};

extern "C" {

int kvc_version(void) { return 3; }

const char* kvc_last_error(void) { return g_last_error.c_str(); }

int kvc_layout_query(int32_t layout, kvc_layout_info* info) {
  if (info == nullptr) return fail(KVC_EINVAL, "kvc_layout_query: info is NULL");
  if (!layout_info(layout, info)) return fail(KVC_EUNSUPPORTED, "kvc_layout_query: unknown layout %d", layout);
  return ok();
}

int kvc_store_rows(const kvc_cache* cache, const void* rows_bf16, int64_t row_stride,
                   const int32_t* out_loc, int64_t n, int32_t* status, void* stream) {
  const char* who = "kvc_store_rows";
  kvc::StoreParams p{};
  int rc = check_cache(cache, &p.cache, who);
  if (rc) return rc;
  if (n < 0) return fail(KVC_EINVAL, "%s: n < 0", who);
  if (n == 0) return ok();
  if (rows_bf16 == nullptr || out_loc == nullptr) return fail(KVC_EINVAL, "%s: NULL rows or out_loc", who);
  if (!aligned16(rows_bf16) || !row_stride_ok(row_stride))
    return fail(KVC_EINVAL, "%s: rows must be 16-byte aligned with row_stride >= 512, a multiple of 8", who);
  p.rows = static_cast<const uint16_t*>(rows_bf16);
  p.row_stride = row_stride;
  p.out_loc = out_loc;
  p.n = n;
  p.status = status;
  return launched(kvc::launch_store_rows(p, static_cast<hipStream_t>(stream)), who);
}

int kvc_store_rows_rope(const kvc_cache* cache, const void* rows_bf16, int64_t row_stride,
                        const int32_t* positions, const float* freqs, int64_t max_pos,
                        const int32_t* out_loc, int64_t n, int32_t* status, void* stream) {
  const char* who = "kvc_store_rows_rope";
  kvc::StoreParams p{};
  int rc = check_cache(cache, &p.cache, who);
  if (rc) return rc;
  if (n < 0) return fail(KVC_EINVAL, "%s: n < 0", who);
  if (n == 0) return ok();
  if (rows_bf16 == nullptr || out_loc == nullptr || positions == nullptr)
    return fail(KVC_EINVAL, "%s: NULL rows, out_loc or positions", who);
  if (!aligned16(rows_bf16) || !row_stride_ok(row_stride))
    return fail(KVC_EINVAL, "%s: rows must be 16-byte aligned with row_stride >= 512, a multiple of 8", who);
  if (freqs == nullptr || !aligned16(freqs) || max_pos < 1)
    return fail(KVC_EINVAL, "%s: freqs must be non-NULL, 16-byte aligned, max_pos >= 1", who);
  p.rows = static_cast<const uint16_t*>(rows_bf16);
  p.row_stride = row_stride;
  p.out_loc = out_loc;
  p.n = n;
  p.status = status;
  p.positions = positions;
  p.freqs = freqs;
  p.max_pos = max_pos;
  return launched(kvc::launch_store_rows(p, static_cast<hipStream_t>(stream)), who);
}

int kvc_dcp_filter_ids(const int32_t* ids, int64_t T, int32_t k, int64_t ids_stride,
                       const int32_t* token_to_req, int32_t n_req, const int32_t* block_table,
                       int64_t bt_stride, int64_t bt_width, const int32_t* valid, int32_t page_size,
                       int64_t num_pages, int32_t world, int32_t rank, int32_t interleave,
                       int32_t* out_slots, int64_t out_stride, int32_t* out_lens,
                       int32_t* status, void* stream) {
  const char* who = "kvc_dcp_filter_ids";
  if (T < 0 || k < 0 || k > 65536) return fail(KVC_EINVAL, "%s: T < 0 or k outside [0, 65536]", who);
  if (T == 0) return ok();
  if (page_size < 1 || page_size > 4096 || (page_size & (page_size - 1)) != 0)
    return fail(KVC_EINVAL, "%s: page_size %d is not a power of two in [1, 4096]", who, page_size);
  if (world < 1 || world > 1024 || rank < 0 || rank >= world)
    return fail(KVC_EINVAL, "%s: world %d / rank %d (1 <= world <= 1024, 0 <= rank < world)", who,
                world, rank);
  if (interleave < 1 || page_size % interleave != 0)
    return fail(KVC_EINVAL, "%s: interleave %d must be >= 1 and divide page_size %d", who,
                interleave, page_size);
  if (token_to_req == nullptr || out_lens == nullptr)
    return fail(KVC_EINVAL, "%s: NULL token_to_req or out_lens", who);
  if (k > 0 && (ids == nullptr || out_slots == nullptr || ids_stride < k || out_stride < k))
    return fail(KVC_EINVAL, "%s: NULL ids or out_slots, or a row stride below k", who);
  if (k > 0 && ((uintptr_t)out_slots & 3u) != 0)
    return fail(KVC_EINVAL, "%s: out_slots is not 4-byte aligned", who);
  if (n_req < 0 || (n_req > 0 && (block_table == nullptr || bt_width < 1 || bt_stride < bt_width)))
    return fail(KVC_EINVAL, "%s: n_req < 0, or no block table, or not 1 <= bt_width <= bt_stride",
                who);
  if (num_pages < 1 || num_pages > ((int64_t)1 << 31) / page_size)
    return fail(KVC_EINVAL, "%s: num_pages must be >= 1 with num_pages * page_size in int32", who);
  kvc::DcpFilterParams p{};
  p.ids = ids;
  p.T = T;
  p.k = k;
  p.ids_stride = ids_stride;
  p.token_to_req = token_to_req;
  p.n_req = n_req;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.bt_width = bt_width;
  p.valid = valid;
  p.page_bits = page_bits_of(page_size);
  p.num_pages = num_pages;
  p.world = world;
  p.world_div = kvc::div_magic((uint32_t)world);
  p.world_log2 = -1;
  if ((world & (world - 1)) == 0) {
    p.world_log2 = 0;
    while ((1 << p.world_log2) < world) ++p.world_log2;
  }
  p.rank = rank;
  p.interleave_log2 = page_bits_of(interleave);
  p.out_slots = out_slots;
  p.out_stride = out_stride;
  p.out_lens = out_lens;
  p.status = status;
  return launched(kvc::launch_dcp_filter(p, static_cast<hipStream_t>(stream)), who);
}

int kvc_dequant_gather(const kvc_cache* cache, const int32_t* page_table, int64_t n_pages,
                       const int32_t* ids, int64_t n, void* out_bf16, int64_t out_row_stride,
                       int32_t* status, void* stream) {
  const char* who = "kvc_dequant_gather";
  kvc::GatherParams p{};
  int rc = check_cache(cache, &p.cache, who);
  if (rc) return rc;
  if (n < 0) return fail(KVC_EINVAL, "%s: n < 0", who);
  if (n == 0) return ok();
  if (ids == nullptr || out_bf16 == nullptr) return fail(KVC_EINVAL, "%s: NULL ids or output", who);
  if (page_table != nullptr && n_pages < 1) return fail(KVC_EINVAL, "%s: page table with n_pages < 1", who);
  if (!aligned16(out_bf16) || !row_stride_ok(out_row_stride) || out_row_stride > (1 << 25))
    return fail(KVC_EINVAL, "%s: output must be 16-byte aligned with out_row_stride in [512, 2^25], "
                            "a multiple of 8", who);
  p.page_table = page_table;
  p.n_pages = page_table ? n_pages : 0;
  p.ids = ids;
  p.n = n;
  p.out = static_cast<uint16_t*>(out_bf16);
  p.out_stride = out_row_stride;
  p.status = status;
  return launched(kvc::launch_dequant_gather(p, static_cast<hipStream_t>(stream)), who);
}

int kvc_compress_store(const kvc_compress_args* a, void* stream) {
  const char* who = "kvc_compress_store";
  if (a == nullptr) return fail(KVC_EINVAL, "%s: args is NULL", who);
  kvc::CompressParams p{};
  int rc = check_cache(&a->cache, &p.cache, who);
  if (rc) return rc;
  if (a->ratio != 1 && a->ratio != 2) return fail(KVC_EUNSUPPORTED, "%s: ratio %d (1 or 2)", who, a->ratio);
  if (a->mode != KVC_MODE_PREFILL && a->mode != KVC_MODE_DECODE && a->mode != KVC_MODE_VERIFY)
    return fail(KVC_EUNSUPPORTED, "%s: mode %d", who, a->mode);
  if (a->mode == KVC_MODE_VERIFY && (a->draft_len < 1 || a->draft_len > 64))
    return fail(KVC_EINVAL, "%s: verify draft_len %d outside [1, 64]", who, a->draft_len);
  if (a->ring_slots < 0 || a->ring_slots > 1024)
    return fail(KVC_EINVAL, "%s: ring_slots %d outside [0, 1024]", who, a->ring_slots);
  const int32_t world = a->dcp_world > 1 ? a->dcp_world : 1;
  if (a->dcp_world < 0 || world > 1024 || a->dcp_rank < 0 || a->dcp_rank >= world)
    return fail(KVC_EINVAL, "%s: dcp_world %d / dcp_rank %d (world <= 1024, 0 <= rank < world)",
                who, a->dcp_world, a->dcp_rank);
  if (world > 1 && (a->dcp_interleave < 1 || a->cache.page_size % a->dcp_interleave != 0))
    return fail(KVC_EINVAL, "%s: dcp_interleave %d must be >= 1 and divide page_size %d", who,
                a->dcp_interleave, a->cache.page_size);
  if (a->num_slots < 0) return fail(KVC_EINVAL, "%s: num_slots < 0", who);
  if (a->tile_rows != 0 && a->tile_rows != 1 && a->tile_rows != 2 && a->tile_rows != 4)
    return fail(KVC_EINVAL, "%s: tile_rows %d (0, 1, 2 or 4)", who, a->tile_rows);
  if (a->num_slots == 0) return ok();
  if (a->mode == KVC_MODE_VERIFY && (int64_t)a->num_slots * a->draft_len > 0x7FFFFFFF)
    return fail(KVC_EINVAL, "%s: num_slots * draft_len must be below 2^31 (token indices are int32)",
                who);
  if (a->mode == KVC_MODE_PREFILL && a->num_slots > kvc::max_prefill_slots())
    return fail(KVC_EINVAL, "%s: prefill num_slots %d > %d", who, a->num_slots, kvc::max_prefill_slots());
  if (a->kv == nullptr || !aligned16(a->kv) || !row_stride_ok(a->kv_stride))
    return fail(KVC_EINVAL, "%s: kv must be non-NULL, 16-byte aligned, kv_stride >= 512 and a multiple of 8", who);
  {
    // decode / verify read token rows 0 .. num_slots * D - 1; prefill checks
    // each slot's rows against kv_rows on the device
    const int64_t need = a->mode == KVC_MODE_PREFILL ? 1
                       : (int64_t)a->num_slots * (a->mode == KVC_MODE_VERIFY ? a->draft_len : 1);
    if (a->kv_rows < need)
      return fail(KVC_EINVAL, "%s: kv_rows %lld, need at least %lld", who, (long long)a->kv_rows,
                  (long long)need);
  }
  if (a->ratio == 2) {
    if (a->score == nullptr || !aligned16(a->score) || a->score_stride < 512 || a->score_stride % 8)
      return fail(KVC_EINVAL, "%s: ratio 2 needs an aligned score buffer with score_stride >= 512, a multiple of 8", who);
    if (a->state == nullptr || !aligned16(a->state))
      return fail(KVC_EINVAL, "%s: ratio 2 needs a 16-byte aligned pending-state buffer", who);
  }
  if (a->start_pos == nullptr) return fail(KVC_EINVAL, "%s: start_pos is NULL", who);
  if (a->mode == KVC_MODE_PREFILL) {
    if (a->offsets == nullptr) return fail(KVC_EINVAL, "%s: prefill needs offsets", who);
    if (a->page_table == nullptr)
      return fail(KVC_EINVAL, "%s: prefill needs a page table", who);
  } else if (a->out_loc == nullptr && a->page_table == nullptr) {
    return fail(KVC_EINVAL, "%s: decode and verify need out_loc or a page table", who);
  }
  if (a->page_table != nullptr && (a->pt_width < 1 || a->pt_stride < a->pt_width))
    return fail(KVC_EINVAL, "%s: page table needs 1 <= pt_width <= pt_stride (%lld, %lld)", who,
                (long long)a->pt_width, (long long)a->pt_stride);
  if (a->norm_w == nullptr || !aligned16(a->norm_w)) return fail(KVC_EINVAL, "%s: norm_w NULL or misaligned", who);
  if (a->freqs == nullptr || !aligned16(a->freqs) || a->max_pos < 1)
    return fail(KVC_EINVAL, "%s: freqs must be non-NULL, 16-byte aligned, max_pos >= 1", who);
  if (a->latent_out == nullptr || !aligned16(a->latent_out) || !row_stride_ok(a->latent_stride))
    return fail(KVC_EINVAL, "%s: latent_out must be aligned with latent_stride >= 512, a multiple of 8", who);
  if (a->max_out_rows < 0) return fail(KVC_EINVAL, "%s: max_out_rows < 0", who);
  if (a->prequant_out != nullptr && (!aligned16(a->prequant_out) || !row_stride_ok(a->prequant_stride)))
    return fail(KVC_EINVAL, "%s: prequant_out misaligned or bad prequant_stride", who);
  if (!(a->eps >= 0.0f)) return fail(KVC_EINVAL, "%s: eps must be >= 0", who);
  p.ratio = a->ratio;
  p.mode = a->mode;
  p.kv = static_cast<const uint16_t*>(a->kv);
  p.kv_stride = a->kv_stride;
  p.score = static_cast<const uint16_t*>(a->score);
  p.score_stride = a->score_stride;
  p.kv_rows = a->kv_rows;
  p.num_slots = a->num_slots;
  p.offsets = a->offsets;
  p.start_pos = a->start_pos;
  p.page_table = a->page_table;
  p.pt_stride = a->page_table ? a->pt_stride : 0;
  p.pt_width = a->page_table ? a->pt_width : 0;
  p.out_loc = a->mode != KVC_MODE_PREFILL ? a->out_loc : nullptr;
  p.state = static_cast<uint16_t*>(a->state);
  p.norm_w = static_cast<const uint16_t*>(a->norm_w);
  p.eps = a->eps;
  p.freqs = a->freqs;
  p.max_pos = a->max_pos;
  p.latent = static_cast<uint16_t*>(a->latent_out);
  p.latent_stride = a->latent_stride;
  p.max_out_rows = a->max_out_rows;
  p.prequant = static_cast<uint16_t*>(a->prequant_out);
  p.prequant_stride = a->prequant_stride;
  p.status = a->status;
  p.draft_len = a->mode == KVC_MODE_VERIFY ? a->draft_len : 1;
  p.ring_slots = a->ring_slots > 1 ? a->ring_slots : 1;
  p.dcp_world = world;
  p.dcp_div = kvc::div_magic((uint32_t)world);
  p.dcp_rank = world > 1 ? a->dcp_rank : 0;
  p.dcp_interleave_log2 = world > 1 ? page_bits_of(a->dcp_interleave) : 0;
  p.tile_rows = a->tile_rows;
  return launched(kvc::launch_compress(p, static_cast<hipStream_t>(stream)), who);
}

// ---------------------------------------------------------------- reuse head
kvc_kvbuf* kvc_kvbuf_create(void) {
  kvc_kvbuf* kb = new (std::nothrow) kvc_kvbuf;
  if (kb) std::memset(kb, 0, sizeof *kb);
  return kb;
}

void kvc_kvbuf_destroy(kvc_kvbuf* kb) { delete kb; }

void kvc_kvbuf_forget(kvc_kvbuf* kb) {
  if (kb) kb->valid = false;
}

void kvc_kvbuf_begin_forward(kvc_kvbuf* kb) {
  if (kb) kb->valid = false;
}

int kvc_dequant_gather_reuse(kvc_kvbuf* kb, const kvc_cache* cache, const int32_t* page_table,
                             int64_t n_pages, const int32_t* ids, int64_t n, void* out_bf16,
                             int64_t out_row_stride, int32_t* status, int32_t* hit,
                             void* stream) {
  const char* who = "kvc_dequant_gather_reuse";
  if (kb == nullptr || hit == nullptr || cache == nullptr)
    return fail(KVC_EINVAL, "%s: NULL kvbuf, hit or cache", who);
  *hit = 0;
  const int64_t np = page_table ? n_pages : 0;
  if (kb->valid && kb->base == cache->base && kb->layout == cache->layout &&
      kb->page_size == cache->page_size && kb->page_stride == cache->page_stride &&
      kb->page_table == page_table && kb->n_pages == np && kb->ids == ids && kb->n == n &&
      kb->out == out_bf16 && kb->out_stride == out_row_stride) {
    *hit = 1;
    return ok();
  }
  kb->valid = false;
  const int rc = kvc_dequant_gather(cache, page_table, n_pages, ids, n, out_bf16, out_row_stride,
                                    status, stream);
  if (rc != KVC_OK) return rc;
  kb->valid = true;
  kb->base = cache->base;
  kb->layout = cache->layout;
  kb->page_size = cache->page_size;
  kb->page_stride = cache->page_stride;
  kb->page_table = page_table;
  kb->n_pages = np;
  kb->ids = ids;
  kb->n = n;
  kb->out = out_bf16;
  kb->out_stride = out_row_stride;
  return KVC_OK;
}

// ---------------------------------------------------------------- slot map
int kvc_slot_map(const kvc_slot_map_args* a, void* stream) {
  const char* who = "kvc_slot_map";
  if (a == nullptr) return fail(KVC_EINVAL, "%s: args is NULL", who);
  if (a->ratio != 1 && a->ratio != 2) return fail(KVC_EUNSUPPORTED, "%s: ratio %d (1 or 2)", who, a->ratio);
  if (!page_size_ok(a->page_size))
    return fail(KVC_EINVAL, "%s: page_size %d is not a power of two in [1, 4096]", who, a->page_size);
  if (a->num_pages < 1 || a->num_pages > ((int64_t)1 << 31) / a->page_size)
    return fail(KVC_EINVAL, "%s: num_pages must be >= 1 with num_pages * page_size in int32", who);
  if (a->num_slots < 0 || a->num_slots > kvc::kMaxSlots)
    return fail(KVC_EINVAL, "%s: num_slots %d outside [0, %d]", who, a->num_slots, kvc::kMaxSlots);
  if (a->max_tokens < 0 || a->max_tokens >= 0x7FFFFFFF || a->n_free < 0 || a->n_free >= 0x7FFFFFFF)
    return fail(KVC_EINVAL, "%s: max_tokens and n_free must lie in [0, 2^31 - 2]", who);
  if (a->token_stride < 0 || (int64_t)a->num_slots * a->token_stride > a->max_tokens)
    return fail(KVC_EINVAL, "%s: token_stride %d: num_slots * token_stride must not pass max_tokens",
                who, a->token_stride);
  if (a->depth != nullptr && a->ratio != 1)
    return fail(KVC_EUNSUPPORTED, "%s: depths need ratio 1 (a cached row per drafted token)", who);
  if (a->num_slots > 0) {
    if (a->lens == nullptr) return fail(KVC_EINVAL, "%s: lens is NULL", who);
    if (a->new_lens == nullptr && a->token_stride == 0)
      return fail(KVC_EINVAL, "%s: new_lens may be NULL only with a token_stride", who);
    if (a->start_pos != nullptr && (a->start_pos == a->lens || a->start_pos == a->new_lens))
      return fail(KVC_EINVAL, "%s: start_pos must not be an input", who);
    if (a->page_table == nullptr || a->pt_width < 1 || a->pt_stride < a->pt_width)
      return fail(KVC_EINVAL, "%s: page table needs 1 <= pt_width <= pt_stride (%lld, %lld)", who,
                  (long long)a->pt_width, (long long)a->pt_stride);
    if (a->n_free > 0 && a->free_pages == nullptr)
      return fail(KVC_EINVAL, "%s: free_pages is NULL with n_free > 0", who);
  }
  if (kvc::launch_slot_map == nullptr) return fail(KVC_ELAUNCH, "%s: built without kernels", who);
  kvc::SlotMapParams p{};
  p.ratio = a->ratio;
  p.page_bits = page_bits_of(a->page_size);
  p.num_pages = a->num_pages;
  p.num_slots = a->num_slots;
  p.token_stride = a->token_stride;
  p.stride_div = kvc::div_magic((uint32_t)(a->token_stride > 0 ? a->token_stride : 1));
  p.lens = a->lens;
  p.new_lens = a->new_lens;
  p.depth = a->depth;
  p.page_table = a->page_table;
  p.pt_stride = a->pt_stride;
  p.pt_width = a->pt_width;
  p.free_pages = a->free_pages;
  p.n_free = a->n_free;
  p.max_tokens = a->max_tokens;
  p.offsets = a->offsets;
  p.start_pos = a->start_pos;
  p.out_loc = a->out_loc;
  p.positions = a->positions;
  p.token_to_req = a->token_to_req;
  p.totals = a->totals;
  p.status = a->status;
  return launched(kvc::launch_slot_map(p, static_cast<hipStream_t>(stream)), who);
}

// --------------------------------------------------------------- attention
int kvc_attend_workspace(int32_t num_slots, int64_t tokens, int32_t num_heads, int64_t* bytes) {
  const char* who = "kvc_attend_workspace";
  if (bytes == nullptr) return fail(KVC_EINVAL, "%s: bytes is NULL", who);
  if (num_slots < 0 || num_slots > kvc::kMaxSlots || num_heads < 1 || num_heads > 1024 || tokens < 0 ||
      tokens > kMaxQueries / num_heads)
    return fail(KVC_EINVAL, "%s: sizes outside those of an attention call", who);
  *bytes = attend_bytes(tokens, num_heads);
  return ok();
}

int kvc_attend_prefill(const kvc_attend_args* args, void* stream) {
  return attend(args, false, stream, "kvc_attend_prefill");
}

int kvc_attend_tree(const kvc_attend_args* args, void* stream) {
  return attend(args, true, stream, "kvc_attend_tree");
}

// ----------------------------------------------------------------- rotary
int kvc_rope_table(const kvc_rope_table_args* a, void* stream) {
  const char* who = "kvc_rope_table";
  if (a == nullptr) return fail(KVC_EINVAL, "%s: args is NULL", who);
  if (a->scaling < KVC_ROPE_NONE || a->scaling > KVC_ROPE_PARTS)
    return fail(KVC_EUNSUPPORTED, "%s: scaling %d", who, a->scaling);
  const int least = a->scaling == KVC_ROPE_BASE ? 4 : 2;
  if (a->rot_dim < least || a->rot_dim > 2 * kvc::kRopeMaxPairs || a->rot_dim % 2 != 0)
    return fail(KVC_EINVAL, "%s: rot_dim %d must be even, in [%d, %d]", who, a->rot_dim, least,
                2 * kvc::kRopeMaxPairs);
  const int64_t end = (int64_t)1 << 31;
  if (a->n < 0 || a->first < 0 || a->first > end || a->n > end - a->first)
    return fail(KVC_EINVAL, "%s: first and n must be >= 0, first + n at most 2^31", who);
  if (!(a->base > 1.0) || !std::isfinite(a->base)) return fail(KVC_EINVAL, "%s: base must be > 1", who);
  if (a->scaling != KVC_ROPE_NONE && !positive(a->factor))
    return fail(KVC_EINVAL, "%s: factor must be > 0", who);
  if (a->scaling == KVC_ROPE_PARTS &&
      (!positive(a->original) || !positive(a->beta_slow) || !(a->beta_fast >= a->beta_slow) ||
       !std::isfinite(a->beta_fast)))
    return fail(KVC_EINVAL, "%s: scaling by parts needs original > 0 and beta_fast >= beta_slow > 0", who);
  if (!positive(a->mscale)) return fail(KVC_EINVAL, "%s: mscale must be > 0", who);
  if (a->n == 0) return ok();
  if (a->freqs == nullptr || !aligned16(a->freqs))
    return fail(KVC_EINVAL, "%s: freqs must be non-NULL, 16-byte aligned", who);
  kvc::RopeTableParams p{};
  rope_speeds(a, p.speed);
  for (int j = 0; j < a->rot_dim / 2; ++j)
    if (!std::isfinite(p.speed[j])) return fail(KVC_EINVAL, "%s: base and factor give no finite speeds", who);
  if (kvc::launch_rope_table == nullptr) return fail(KVC_ELAUNCH, "%s: built without kernels", who);
  p.freqs = a->freqs;
  p.n = a->n;
  p.first = a->first;
  p.pairs = a->rot_dim / 2;
  p.mscale = a->mscale;
  return launched(kvc::launch_rope_table(p, static_cast<hipStream_t>(stream)), who);
}

int kvc_rope_rows(const kvc_rope_args* a, void* stream) {
  const char* who = "kvc_rope_rows";
  if (a == nullptr) return fail(KVC_EINVAL, "%s: args is NULL", who);
  if (a->dtype < KVC_BF16 || a->dtype > KVC_FP32) return fail(KVC_EUNSUPPORTED, "%s: dtype %d", who, a->dtype);
  if (a->num_heads < 1 || a->num_heads > 1024)
    return fail(KVC_EINVAL, "%s: num_heads %d outside [1, 1024]", who, a->num_heads);
  if (a->head_dim < 2 || a->head_dim > 8192)
    return fail(KVC_EINVAL, "%s: head_dim %d outside [2, 8192]", who, a->head_dim);
  if (a->rot_dim < 2 || a->rot_dim > a->head_dim || a->rot_dim % 2 != 0)
    return fail(KVC_EINVAL, "%s: rot_dim %d must be even, in [2, head_dim]", who, a->rot_dim);
  if (a->offset < 0 || a->offset > a->head_dim - a->rot_dim)
    return fail(KVC_EINVAL, "%s: offset %d outside [0, head_dim - rot_dim]", who, a->offset);
  if (a->tokens < 0 || a->tokens > 0x7FFFFFFF) return fail(KVC_EINVAL, "%s: tokens outside [0, 2^31)", who);
  if (a->max_pos < 1) return fail(KVC_EINVAL, "%s: max_pos must be >= 1", who);
  if (a->tokens == 0) return ok();
  const uintptr_t size = a->dtype == KVC_FP32 ? 4 : 2;
  if (a->x == nullptr || a->out == nullptr || (uintptr_t)a->x % size != 0 || (uintptr_t)a->out % size != 0)
    return fail(KVC_EINVAL, "%s: x and out must be non-NULL and aligned to their type", who);
  kvc::RopeRowsParams p{};
  // (the stride of an axis of one entry is not used)
  p.x_stride = a->tokens > 1 ? a->x_stride : 0;
  p.x_hstride = a->num_heads > 1 ? a->x_head_stride : 0;
  p.out_stride = a->tokens > 1 ? a->out_stride : 0;
  p.out_hstride = a->num_heads > 1 ? a->out_head_stride : 0;
  if (p.x_stride < 0 || p.x_hstride < 0) return fail(KVC_EINVAL, "%s: x strides must be >= 0", who);
  if ((a->tokens > 1 && p.out_stride < a->head_dim) || (a->num_heads > 1 && p.out_hstride < a->head_dim))
    return fail(KVC_EINVAL, "%s: out strides must be >= head_dim", who);
  p.in_place = a->x == a->out;
  if (p.in_place && (p.x_stride != p.out_stride || p.x_hstride != p.out_hstride))
    return fail(KVC_EINVAL, "%s: out is x, with other strides", who);
  if (a->positions == nullptr || a->freqs == nullptr || (uintptr_t)a->freqs % 8 != 0)
    return fail(KVC_EINVAL, "%s: NULL positions or freqs, or freqs not 8-byte aligned", who);
  if (kvc::launch_rope_rows == nullptr) return fail(KVC_ELAUNCH, "%s: built without kernels", who);
  p.x = a->x;
  p.out = a->out;
  p.tokens = a->tokens;
  p.heads = a->num_heads;
  p.dim = a->head_dim;
  p.rot = a->rot_dim;
  p.offset = a->offset;
  p.type = a->dtype;
  p.half = a->half != 0;
  p.transpose = a->transpose != 0;
  p.positions = a->positions;
  p.freqs = a->freqs;
  p.max_pos = a->max_pos;
  p.status = a->status;
  return launched(kvc::launch_rope_rows(p, static_cast<hipStream_t>(stream)), who);
}

// --------------------------------------------------------------- eviction
int kvc_weigh_workspace(int64_t* bytes) {
  if (bytes == nullptr) return fail(KVC_EINVAL, "kvc_weigh_workspace: bytes is NULL");
  *bytes = kWeighBytes;
  return ok();
}

int kvc_weigh_prefill(const kvc_weigh_args* args, void* stream) {
  return weigh(args, false, stream, "kvc_weigh_prefill");
}

int kvc_weigh_tree(const kvc_weigh_args* args, void* stream) {
  return weigh(args, true, stream, "kvc_weigh_tree");
}

int kvc_evict_workspace(int32_t num_slots, int64_t w_width, int64_t* bytes) {
  const char* who = "kvc_evict_workspace";
  if (bytes == nullptr) return fail(KVC_EINVAL, "%s: bytes is NULL", who);
  if (num_slots < 0 || num_slots > kvc::kMaxSlots || w_width < 1)
    return fail(KVC_EINVAL, "%s: sizes outside those of a call", who);
  *bytes = evict_bytes(num_slots, w_width);
  return ok();
}

int kvc_evict_select(const kvc_evict_args* a, void* stream) {
  const char* who = "kvc_evict_select";
  if (a == nullptr) return fail(KVC_EINVAL, "%s: args is NULL", who);
  if (a->ratio != 1 && a->ratio != 2) return fail(KVC_EUNSUPPORTED, "%s: ratio %d (1 or 2)", who, a->ratio);
  if (a->num_slots < 0 || a->num_slots > kvc::kMaxSlots)
    return fail(KVC_EINVAL, "%s: num_slots %d outside [0, %d]", who, a->num_slots, kvc::kMaxSlots);
  if (a->first < 0 || a->recent < 0) return fail(KVC_EINVAL, "%s: first and recent must be >= 0", who);
  if (a->num_slots == 0) return ok();
  if (a->lens == nullptr || a->counts == nullptr || a->counts == a->lens)
    return fail(KVC_EINVAL, "%s: NULL lens or counts, or counts is lens", who);
  if (a->weights == nullptr || a->w_width < 1 || a->w_stride < a->w_width)
    return fail(KVC_EINVAL, "%s: weights need 1 <= w_width <= w_stride (%lld, %lld)", who,
                (long long)a->w_width, (long long)a->w_stride);
  if (a->kept == nullptr || a->kept_width < 1 || a->kept_width > 0x7FFFFFFF || a->kept_stride < a->kept_width)
    return fail(KVC_EINVAL, "%s: kept needs 1 <= kept_width <= kept_stride (%lld, %lld)", who,
                (long long)a->kept_width, (long long)a->kept_stride);
  if (a->kept_weights != nullptr && (a->kw_stride < a->kept_width || a->kept_weights == a->weights))
    return fail(KVC_EINVAL, "%s: kept_weights needs a stride >= kept_width, and is not weights", who);
  const int32_t segments = evict_segments(a->num_slots, a->w_width);
  const int64_t all = (int64_t)segments * a->num_slots;
  const int64_t need = all * (3 * kvc::kSelectWords + 4) * 4;
  if (need > 0 && (a->workspace == nullptr || ((uintptr_t)a->workspace & 255u) != 0 || a->workspace_bytes < need))
    return fail(KVC_EINVAL, "%s: workspace needs %lld bytes, 256-byte aligned", who, (long long)need);
  if (kvc::launch_select == nullptr) return fail(KVC_ELAUNCH, "%s: built without kernels", who);
  kvc::SelectParams p{};
  p.ratio = a->ratio;
  p.num_slots = a->num_slots;
  p.lens = a->lens;
  p.weights = a->weights;
  p.w_stride = a->w_stride;
  p.w_width = a->w_width;
  p.budget = a->budget;
  p.budgets = a->budgets;
  p.first = a->first;
  p.recent = a->recent;
  p.kept = a->kept;
  p.kept_stride = a->kept_stride;
  p.kept_width = (int32_t)a->kept_width;
  p.counts = a->counts;
  p.kept_weights = a->kept_weights;
  p.kw_stride = a->kw_stride;
  p.status = a->status;
  if (segments > 0) {
    p.segments = segments;
    p.segment_rows = (a->w_width - 1) / segments + 1;
    p.hists = static_cast<uint32_t*>(a->workspace);
    p.states = reinterpret_cast<int32_t*>(p.hists + 3 * all * kvc::kSelectWords);
  }
  return launched(kvc::launch_select(p, static_cast<hipStream_t>(stream)), who);
}

int kvc_cache_compact(const kvc_compact_args* a, void* stream) {
  const char* who = "kvc_cache_compact";
  if (a == nullptr) return fail(KVC_EINVAL, "%s: args is NULL", who);
  kvc::CompactParams p{};
  int rc = check_cache(&a->cache, &p.cache, who);
  if (rc) return rc;
  if (a->ratio != 1 && a->ratio != 2) return fail(KVC_EUNSUPPORTED, "%s: ratio %d (1 or 2)", who, a->ratio);
  if (a->num_slots < 0 || a->num_slots > kvc::kMaxSlots)
    return fail(KVC_EINVAL, "%s: num_slots %d outside [0, %d]", who, a->num_slots, kvc::kMaxSlots);
  if (a->n_free < 0 || a->n_free >= 0x7FFFFFFF || a->freed_cap < 0 || a->freed_cap >= 0x7FFFFFFF)
    return fail(KVC_EINVAL, "%s: n_free and freed_cap must lie in [0, 2^31 - 2]", who);
  if (a->num_slots == 0) {
    if (a->totals == nullptr) return ok();
    if (kvc::launch_compact == nullptr) return fail(KVC_ELAUNCH, "%s: built without kernels", who);
    p.ratio = a->ratio;
    p.totals = a->totals;
    return launched(kvc::launch_compact(p, static_cast<hipStream_t>(stream)), who);
  }
  if (a->lens == nullptr || a->counts == nullptr || a->new_lens == nullptr)
    return fail(KVC_EINVAL, "%s: NULL lens, counts or new_lens", who);
  if (a->new_lens == a->lens || a->new_lens == a->counts)
    return fail(KVC_EINVAL, "%s: new_lens must not be an input", who);
  if (a->kept == nullptr || a->kept_width < 1 || a->kept_width > 0x7FFFFFFF || a->kept_stride < a->kept_width)
    return fail(KVC_EINVAL, "%s: kept needs 1 <= kept_width <= kept_stride (%lld, %lld)", who,
                (long long)a->kept_width, (long long)a->kept_stride);
  if (a->page_table == nullptr || a->pt_width < 1 || a->pt_stride < a->pt_width)
    return fail(KVC_EINVAL, "%s: page table needs 1 <= pt_width <= pt_stride (%lld, %lld)", who,
                (long long)a->pt_width, (long long)a->pt_stride);
  if (a->new_table == nullptr || a->nt_stride < a->pt_width || a->new_table == a->page_table)
    return fail(KVC_EINVAL, "%s: new_table needs a stride >= pt_width, and is not page_table", who);
  if (a->n_free > 0 && a->free_pages == nullptr)
    return fail(KVC_EINVAL, "%s: free_pages is NULL with n_free > 0", who);
  if (a->freed != nullptr && a->freed == a->free_pages)
    return fail(KVC_EINVAL, "%s: freed must not be free_pages", who);
  if ((a->kept_weights == nullptr) != (a->weights == nullptr))
    return fail(KVC_EINVAL, "%s: kept_weights and weights come together", who);
  if (a->weights != nullptr && (a->kw_stride < a->kept_width || a->w_width < 1 || a->w_stride < a->w_width ||
                                a->weights == a->kept_weights))
    return fail(KVC_EINVAL, "%s: weights need 1 <= w_width <= w_stride, kept_weights a stride >= kept_width, "
                            "and memory of its own", who);
  if (kvc::launch_compact == nullptr) return fail(KVC_ELAUNCH, "%s: built without kernels", who);
  p.ratio = a->ratio;
  p.num_slots = a->num_slots;
  p.lens = a->lens;
  p.kept = a->kept;
  p.kept_stride = a->kept_stride;
  p.kept_width = (int32_t)a->kept_width;
  p.counts = a->counts;
  p.page_table = a->page_table;
  p.pt_stride = a->pt_stride;
  p.pt_width = a->pt_width;
  p.free_pages = a->free_pages;
  p.n_free = a->n_free;
  p.new_table = a->new_table;
  p.nt_stride = a->nt_stride;
  p.new_lens = a->new_lens;
  p.kept_weights = a->kept_weights;
  p.kw_stride = a->kw_stride;
  p.weights = a->weights;
  p.w_stride = a->w_stride;
  p.w_width = a->w_width;
  p.freed = a->freed;
  p.freed_cap = a->freed_cap;
  p.totals = a->totals;
  p.status = a->status;
  return launched(kvc::launch_compact(p, static_cast<hipStream_t>(stream)), who);
}

}  // extern "C"
