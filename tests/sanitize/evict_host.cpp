// evict_host.cpp -- the host code of the rotary calls and the eviction up to and
// past their launches, under AddressSanitizer and UBSan.  The launchers here
// take the arguments and launch nothing; main checks what they were given:
// workspaces' parts lie apart inside the bytes asked for, segments cover a row of
// weights, strides of single entries are not looked at, speeds are finite.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <limits>

#include "../../fp8_fp4_quantized_amd/csrc/launch_evict.hpp"
#include "../../include/kvc.h"

namespace {
kvc::RopeTableParams g_table;
kvc::RopeRowsParams g_rows;
kvc::WeighParams g_weigh;
kvc::SelectParams g_select;
kvc::CompactParams g_compact;
int64_t g_queries;
int g_launches;
}  // namespace

namespace kvc {
hipError_t launch_store_rows(const StoreParams&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_dequant_gather(const GatherParams&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_compress(const CompressParams&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_dcp_filter(const DcpFilterParams&, hipStream_t) { return hipErrorNoDevice; }
int max_prefill_slots() { return 8191; }
hipError_t launch_rope_table(const RopeTableParams& p, hipStream_t) {
  g_table = p;
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_rope_rows(const RopeRowsParams& p, hipStream_t) {
  g_rows = p;
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_weigh(const WeighParams& p, int64_t slot_queries, hipStream_t) {
  g_weigh = p;
  g_queries = slot_queries;
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_select(const SelectParams& p, hipStream_t) {
  g_select = p;
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_compact(const CompactParams& p, hipStream_t) {
  g_compact = p;
  ++g_launches;
  return hipSuccess;
}
}  // namespace kvc

#define CHECK(c)                                                                          \
  do {                                                                                    \
    if (!(c)) {                                                                           \
      std::printf("line %d: %s (%lld, %lld, %lld): %s\n", __LINE__, #c, (long long)one,   \
                  (long long)two, (long long)three, kvc_last_error());                    \
      return 1;                                                                           \
    }                                                                                     \
  } while (0)

namespace {

// pointers that the host code passes on and must not follow
template <typename T = void>
T* fake(uintptr_t n) { return reinterpret_cast<T*>(0x7F0000000000u + (n << 32)); }
// the kernels' division by a number that the host prepared
uint32_t quotient(uint32_t n, const kvc::DivMagic& d) {
  const uint32_t t = (uint32_t)((uint64_t)d.m * n >> 32);
  return (t + ((n - t) >> d.sh1)) >> d.sh2;
}
const uint8_t* bytes_of(const void* p) { return static_cast<const uint8_t*>(p); }

int weigh(int32_t one /* slots */, int64_t two /* tokens a slot */, int32_t three /* heads */, bool tree) {
  kvc_weigh_args a{};
  a.ratio = 1;
  a.num_heads = three;
  a.num_slots = one;
  a.draft_len = tree ? (int32_t)two : -7;
  a.q = fake(1);
  a.q_stride = (int64_t)three * 512;
  a.q_head_stride = three > 1 ? 512 : -3;               // (of one head: not looked at)
  a.q_rows = tree ? one * two : two;
  a.lse = fake<float>(2);
  a.offsets = fake<int32_t>(3);
  a.start_pos = fake<int32_t>(4);
  a.page_table = fake<int32_t>(5);
  a.pt_stride = a.pt_width = std::numeric_limits<int64_t>::max();
  a.scale = 0.05f;
  a.decay = 0.5f;
  a.prev = a.weights = fake<float>(6);
  a.prev_stride = a.w_stride = 2000;
  a.w_width = 1000;
  a.cache = kvc_cache{fake(7), KVC_LAYOUT_V41, 64, 64 * 528, 10};
  int64_t need = -1;
  CHECK(kvc_weigh_workspace(&need) == KVC_OK && need > 0);
  const int64_t queries = two * three;
  auto call = [&] { return tree ? kvc_weigh_tree(&a, nullptr) : kvc_weigh_prefill(&a, nullptr); };
  const int before = g_launches;
  if (one > 0 && two > 0 && queries > kvc::kWeighFew) {
    CHECK(call() == KVC_EINVAL);
    a.workspace = fake(8);
    a.workspace_bytes = need - 1;
    CHECK(call() == KVC_EINVAL && g_launches == before);
    a.workspace_bytes = need;
  }
  CHECK(call() == KVC_OK);
  if (one == 0 || two == 0) {
    CHECK(g_launches == before);
    return 0;
  }
  CHECK(g_launches == before + 1 && g_queries == queries);
  const kvc::WeighParams& p = g_weigh;
  CHECK(p.pt_width == 0x7FFFFFFF && p.prev == a.prev && (p.offsets == nullptr) == tree);
  CHECK(p.draft_len == (tree ? a.draft_len : 0) && (three > 1 || p.q_hstride == 0));
  for (uint32_t n : {0u, 1u, (uint32_t)three - 1, (uint32_t)three, 0x7FFFFEFFu})
    CHECK(quotient(n, p.head_div) == n / (uint32_t)three);
  if (queries > kvc::kWeighFew) {
    CHECK(bytes_of(p.head) == bytes_of(a.workspace) && bytes_of(p.parts) >= bytes_of(p.head + 1));
    CHECK(bytes_of(p.parts + (int64_t)kvc::kWeighParts * kvc::kWeighRows) <= bytes_of(a.workspace) + need);
    CHECK((reinterpret_cast<uintptr_t>(p.parts) & 255) == 0);
  } else {
    CHECK(p.head == nullptr && p.parts == nullptr);
  }
  a.decay = 0.0f;
  CHECK(call() == KVC_OK && g_weigh.prev == nullptr);
  // one slot has no next row
  a.prev_stride = 1500;
  CHECK(call() == (one > 1 ? KVC_EINVAL : KVC_OK));
  return 0;
}

int select(int32_t one /* slots */, int64_t two /* weights a row */) {
  const int three = 0;
  kvc_evict_args a{};
  a.ratio = 1;
  a.num_slots = one;
  a.lens = fake<int32_t>(1);
  a.weights = fake<float>(2);
  a.w_stride = a.w_width = two;
  a.budget = 5;
  a.kept = fake<int32_t>(3);
  a.kept_stride = a.kept_width = 0x7FFFFFFF;
  a.counts = fake<int32_t>(4);
  int64_t need = -1;
  CHECK(kvc_evict_workspace(one, two, &need) == KVC_OK && need >= 0);
  const uint8_t* const w = fake<uint8_t>(5);
  a.workspace = need > 0 ? fake(5) : nullptr;
  a.workspace_bytes = need;
  const int before = g_launches;
  CHECK(kvc_evict_select(&a, nullptr) == KVC_OK);
  if (one == 0) {
    CHECK(g_launches == before);
    return 0;
  }
  CHECK(g_launches == before + 1);
  const kvc::SelectParams& p = g_select;
  CHECK(p.kept_width == 0x7FFFFFFF && p.w_width == two);
  if (p.segments == 0) {
    CHECK(two <= kvc::kSelectRegisterRows || one > kvc::kSelectSegmentSlots);
    CHECK(p.hists == nullptr && p.states == nullptr);
    return 0;
  }
  const int64_t all = (int64_t)p.segments * one;
  CHECK(two > kvc::kSelectRegisterRows && all <= kvc::kSelectSegments && p.segments <= 65535);
  // the segments cover the row, and none is without any of it
  CHECK(p.segment_rows > (two - 1) / p.segments && p.segment_rows <= (two - 1) / p.segments + 1);
  CHECK((two - 1) / p.segment_rows + 1 <= p.segments);
  CHECK(bytes_of(p.hists) == w && bytes_of(p.states) >= bytes_of(p.hists + 3 * all * kvc::kSelectWords));
  CHECK(bytes_of(p.states + 4 * all) <= w + need);
  a.workspace_bytes = (bytes_of(p.states + 4 * all) - w) - 1;
  CHECK(kvc_evict_select(&a, nullptr) == KVC_EINVAL && g_launches == before + 1);
  return 0;
}

int compact(int32_t one /* slots */, int64_t two /* pages a table row */) {
  const int three = 0;
  kvc_compact_args a{};
  a.ratio = 2;
  a.num_slots = one;
  a.lens = fake<int32_t>(1);
  a.kept = fake<int32_t>(2);
  a.kept_stride = a.kept_width = 0x7FFFFFFF;
  a.counts = fake<int32_t>(3);
  a.page_table = fake<int32_t>(4);
  a.pt_stride = a.pt_width = two;
  a.n_free = 0;
  a.new_table = fake<int32_t>(6);
  a.nt_stride = two;
  a.new_lens = fake<int32_t>(7);
  a.cache = kvc_cache{fake(8), KVC_LAYOUT_V41_FP4, 1, 288, (int64_t(1) << 31)};
  const int before = g_launches;
  CHECK(kvc_cache_compact(&a, nullptr) == KVC_OK);
  CHECK(g_launches == before + (one > 0 ? 1 : 0));
  a.totals = fake<int32_t>(9);
  CHECK(kvc_cache_compact(&a, nullptr) == KVC_OK && g_compact.totals == a.totals && g_compact.num_slots == one);
  CHECK(g_compact.weights == nullptr && g_compact.freed == nullptr && g_compact.n_free == 0);
  CHECK(one == 0 || (g_compact.kept_width == 0x7FFFFFFF && g_compact.pt_width == two && g_compact.cache.page_bits == 0));
  if (one == 0) return 0;
  a.freed = fake<int32_t>(10);
  a.freed_cap = 0x7FFFFFFE;
  a.free_pages = fake<int32_t>(5);
  a.n_free = 0x7FFFFFFE;
  a.kept_weights = fake<float>(11);
  a.kw_stride = 0x7FFFFFFF;
  a.weights = fake<float>(12);
  a.w_stride = a.w_width = 1;
  CHECK(kvc_cache_compact(&a, nullptr) == KVC_OK && g_compact.freed_cap == 0x7FFFFFFE && g_compact.w_width == 1);
  return 0;
}

int table(int32_t one /* scaling */, int32_t two /* rot_dim */, double base, double factor, double original,
          double fast) {
  const int three = 0;
  kvc_rope_table_args a{};
  a.freqs = fake<float>(1);
  a.n = 1;
  a.first = 0x7FFFFFFF;
  a.rot_dim = two;
  a.scaling = one;
  a.base = base;
  a.factor = factor;
  a.original = original;
  a.beta_fast = fast;
  a.beta_slow = 1.0;
  a.mscale = 1.0;
  const int before = g_launches;
  const int rc = kvc_rope_table(&a, nullptr);
  CHECK(rc == KVC_OK || rc == KVC_EINVAL);
  if (rc != KVC_OK) {
    CHECK(g_launches == before);
    return 0;
  }
  CHECK(g_launches == before + 1 && g_table.pairs == two / 2 && g_table.first == a.first);
  for (int j = 0; j < g_table.pairs; ++j) {
    CHECK(std::isfinite(g_table.speed[j]) && g_table.speed[j] >= 0);
    // (a base made less than 1 by its factor turns later pairs faster)
    CHECK(j == 0 || one == KVC_ROPE_PARTS || factor < 1 || g_table.speed[j] <= g_table.speed[j - 1]);
  }
  return 0;
}

int rows(int32_t one /* tokens */, int32_t two /* heads */, int32_t three /* in place */) {
  kvc_rope_args a{};
  a.dtype = KVC_BF16;
  a.num_heads = two;
  a.head_dim = 8192;
  a.rot_dim = 64;
  a.offset = 8192 - 64;
  a.half = 17;
  a.transpose = -1;
  a.tokens = one;
  a.x = fake(1);
  a.x_stride = one > 1 ? two * int64_t(8192) : -1;      // (of one token, or head: not looked at)
  a.x_head_stride = two > 1 ? 8192 : std::numeric_limits<int64_t>::min();
  a.out = three ? fake(1) : fake(2);
  a.out_stride = one > 1 ? two * int64_t(8192) : 3;
  a.out_head_stride = two > 1 ? 8192 : 0;
  a.positions = fake<int32_t>(3);
  a.freqs = fake<float>(4);
  a.max_pos = std::numeric_limits<int64_t>::max();
  const int before = g_launches;
  CHECK(kvc_rope_rows(&a, nullptr) == KVC_OK);
  CHECK(g_launches == before + (one > 0 ? 1 : 0));
  if (one == 0) return 0;
  CHECK(g_rows.in_place == three && g_rows.half == 1 && g_rows.transpose == 1);
  CHECK(g_rows.x_stride == (one > 1 ? a.x_stride : 0) && g_rows.out_hstride == (two > 1 ? 8192 : 0));
  return 0;
}

}  // namespace

int main() {
  int n = 0;
  for (int heads : {1, 3, 16, 64, 128, 129, 1024})
    for (int slots : {0, 1, 2, 255, 8191}) {
      for (int64_t tokens : {int64_t(0), int64_t(1), int64_t(2), int64_t(128), int64_t(0x7FFFFF00) / heads}) {
        if (weigh(slots, tokens, heads, false)) return 1;
        ++n;
      }
      for (int draft : {1, 2, 64}) {
        if ((int64_t)slots * draft > 0x7FFFFF00 / heads) continue;
        if (weigh(slots, draft, heads, true)) return 1;
        ++n;
      }
    }
  const int64_t top = std::numeric_limits<int64_t>::max();
  for (int slots : {0, 1, 2, 3, 31, 64, 127, 128, 129, 8191})
    for (int64_t width : {int64_t(1), int64_t(32768), int64_t(32769), int64_t(49153), int64_t(100000), int64_t(1) << 20,
                          (int64_t(1) << 23) + 1, (int64_t(1) << 31) - 1, int64_t(1) << 40, top}) {
      if (select(slots, width)) return 1;
      ++n;
    }
  for (int slots : {0, 1, 8191})
    for (int64_t width : {int64_t(1), int64_t(1) << 31}) {
      if (compact(slots, width)) return 1;
      ++n;
    }
  for (int scaling : {0, 1, 2, 3})
    for (int rot : {2, 4, 6, 510, 512})
      for (double base : {std::nextafter(1.0, 2.0), 2.0, 1e4, 1e300})
        for (double factor : {5e-324, 1e-3, 1.0, 32.0, 1e308})
          for (double original : {5e-324, 1.0, 4096.0, 1e308})
            for (double fast : {1.0, 32.0, 1e308}) {
              if (table(scaling, rot, base, factor, original, fast)) return 1;
              ++n;
            }
  for (int tokens : {0, 1, 2, 0x7FFFFFFF})
    for (int heads : {1, 2, 1024})
      for (int in_place : {0, 1}) {
        if (rows(tokens, heads, in_place)) return 1;
        ++n;
      }
  std::printf("%d calls, all checks passed\n", n);
  return 0;
}
