// attend_host.cpp -- the host code of the attention and the slot map up to and
// past their launches, under AddressSanitizer and UBSan.  The launchers here
// take the arguments and launch nothing; main checks what they were given: the
// workspace's parts lie apart inside the bytes asked for and hold what the
// kernels write there, and the units agree with a count of them one by one.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../fp8_fp4_quantized_amd/csrc/launch_attend.hpp"
#include "../../include/kvc.h"

namespace {
kvc::AttendParams g_attend;
kvc::SlotMapParams g_map;
int g_qblocks, g_launches;
}  // namespace

namespace kvc {
hipError_t launch_store_rows(const StoreParams&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_dequant_gather(const GatherParams&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_compress(const CompressParams&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_dcp_filter(const DcpFilterParams&, hipStream_t) { return hipErrorNoDevice; }
int max_prefill_slots() { return 8191; }
hipError_t launch_attend(const AttendParams& p, int qblocks, hipStream_t) {
  g_attend = p;
  g_qblocks = qblocks;
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_slot_map(const SlotMapParams& p, hipStream_t) {
  g_map = p;
  ++g_launches;
  return hipSuccess;
}
}  // namespace kvc

#define CHECK(c)                                                            \
  do {                                                                      \
    if (!(c)) {                                                             \
      std::printf("line %d: %s (slots %d, tokens %lld, heads %d, page %d, tree %d)\n", __LINE__, #c, slots, \
                  (long long)tokens, heads, page, (int)tree);               \
      return 1;                                                             \
    }                                                                       \
  } while (0)

namespace {

// pointers that the host code passes on and must not follow
void* fake(uintptr_t n) { return reinterpret_cast<void*>(0x7F0000000000u + (n << 32)); }

int attend(int slots, int64_t tokens, int heads, int page, bool tree, int draft) {
  kvc_attend_args a{};
  a.ratio = 1;
  a.num_heads = heads;
  a.num_slots = slots;
  a.draft_len = draft;
  a.q = fake(1);
  a.q_stride = (int64_t)heads * 512;
  a.q_head_stride = 512;
  a.q_rows = tokens;
  a.offsets = static_cast<const int32_t*>(fake(2));
  a.start_pos = static_cast<const int32_t*>(fake(3));
  a.page_table = static_cast<const int32_t*>(fake(4));
  a.pt_stride = a.pt_width = 100;
  a.scale = 0.05f;
  a.out = fake(5);
  a.out_stride = a.q_stride;
  a.out_head_stride = 512;
  a.cache = kvc_cache{fake(6), KVC_LAYOUT_V41, page, (int64_t)page * 528, 10};
  int64_t bytes = -1;
  const int64_t rows = tree ? (int64_t)slots * draft : tokens;
  CHECK(kvc_attend_workspace(slots, rows, heads, &bytes) == KVC_OK);
  uint8_t* const w = static_cast<uint8_t*>(fake(7));
  a.workspace = w;
  a.workspace_bytes = bytes;
  auto call = [&] { return tree ? kvc_attend_tree(&a, nullptr) : kvc_attend_prefill(&a, nullptr); };
  const int before = g_launches;
  CHECK(call() == KVC_OK);
  if (slots == 0 || tokens == 0) {
    CHECK(g_launches == before);
    return 0;
  }
  CHECK(g_launches == before + 1);
  const kvc::AttendParams& p = g_attend;
  CHECK(g_qblocks == 1 || g_qblocks == 2 || g_qblocks == 4);
  CHECK(page >= 8 || g_qblocks < 4);
  // the parts, in order, apart and inside
  const int64_t parts = 2 * 256 * 32 * (int64_t)g_qblocks;
  const struct { const void* at; int64_t n; } part[] = {
      {p.head, sizeof(kvc::AttendHead)}, {p.starts, (256 + 1) * (int64_t)sizeof(kvc::AttendStart)},
      {p.splits, kvc::kAttendPlanUnits * (int64_t)sizeof(kvc::AttendSplit)}, {p.part_ml, parts * 16},
      {p.part_o, parts * 512 * 4}};
  const uint8_t* end = w;
  for (const auto& x : part) {
    const uint8_t* at = static_cast<const uint8_t*>(x.at);
    CHECK(at >= end && (reinterpret_cast<uintptr_t>(at) & 255) == 0);
    end = at + x.n;
  }
  CHECK(end <= w + bytes);
  // units: of a slot with n tokens, and the most of any split of the tokens
  const int64_t qt = 32 * g_qblocks;
  auto units = [&](int64_t n) { return (n * heads + qt - 1) / qt; };
  const int64_t of_slot = units(tree ? draft : tokens);
  if (p.plan_units > 0) {
    CHECK(p.plan_units == of_slot && of_slot * slots <= kvc::kAttendPlanUnits);
  } else {
    CHECK(of_slot * slots > kvc::kAttendPlanUnits);
  }
  int64_t all = 0, left = rows;
  if (tree) {
    all = units(draft) * slots;
  } else {
    for (int b = 0; b < slots; ++b) {             // a token each, the rest in the last
      const int64_t n = b + 1 < slots ? (left > 1 ? 1 : left) : left;
      all += units(n);
      left -= n;
    }
  }
  CHECK(p.units_max >= all);
  // a byte less is refused
  a.workspace_bytes = bytes - 1;
  CHECK(call() == KVC_EINVAL && g_launches == before + 1);
  return 0;
}

int slot_map() {
  const int slots = 8191, heads = 0, page = 64;
  const int64_t tokens = 0x7FFFFFFE;
  const bool tree = false;
  kvc_slot_map_args a{};
  a.ratio = 2;
  a.page_size = page;
  a.num_pages = (int64_t(1) << 31) / page;
  a.num_slots = slots;
  a.token_stride = (int32_t)(tokens / slots);
  a.lens = static_cast<const int32_t*>(fake(1));
  a.page_table = static_cast<int32_t*>(fake(2));
  a.pt_stride = a.pt_width = int64_t(1) << 40;
  a.free_pages = static_cast<const int32_t*>(fake(3));
  a.n_free = 0x7FFFFFFE;
  a.max_tokens = tokens;
  CHECK(kvc_slot_map(&a, nullptr) == KVC_OK);
  CHECK(g_map.page_bits == 6 && g_map.num_slots == slots && g_map.max_tokens == tokens);
  a.token_stride += 1;
  CHECK(kvc_slot_map(&a, nullptr) == KVC_EINVAL);
  return 0;
}

}  // namespace

int main() {
  int n = 0;
  for (int heads : {1, 3, 8, 16, 64, 65, 128, 1024})
    for (int slots : {0, 1, 2, 7, 64, 255, 256, 257, 8191})
      for (int page : {1, 4, 8, 64, 4096}) {
        for (int64_t tokens : {int64_t(0), int64_t(1), int64_t(33), int64_t(8191), int64_t(70001),
                               int64_t(0x7FFFFF00) / heads}) {
          if (attend(slots, tokens, heads, page, false, 0)) return 1;
          ++n;
        }
        for (int draft : {1, 2, 7, 64}) {
          if ((int64_t)slots * draft > 0x7FFFFF00 / heads) continue;
          if (attend(slots, (int64_t)slots * draft, heads, page, true, draft)) return 1;
          ++n;
        }
      }
  if (slot_map()) return 1;
  std::printf("%d calls, all checks passed\n", n);
  return 0;
}
