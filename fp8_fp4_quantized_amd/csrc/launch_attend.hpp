// launch_attend.hpp -- arguments and launchers of the slot map and the
// attention over the paged cache.
#pragma once

#include "launch.hpp"

namespace kvc {

// status bit of the slot map (beside those of layout.hpp): no free page left
constexpr int32_t kStNoPage = 128;

// largest num_slots of the slot map and of an attention call (their LDS tables)
constexpr int32_t kMaxSlots = 8191;

struct SlotMapParams {
  int32_t ratio;
  int32_t page_bits;
  int64_t num_pages;
  int32_t num_slots;
  int32_t token_stride;        // 0: packed tokens; else rows per slot
  DivMagic stride_div;         // division by token_stride (when > 0)
  const int32_t* lens;
  const int32_t* new_lens;     // NULL: token_stride for every slot
  const int32_t* depth;        // nullable
  int32_t* page_table;
  int64_t pt_stride;
  int64_t pt_width;
  const int32_t* free_pages;
  int64_t n_free;
  int64_t max_tokens;
  int32_t* offsets;            // outputs, each nullable
  int32_t* start_pos;
  int32_t* out_loc;
  int32_t* positions;
  int32_t* token_to_req;
  int32_t* totals;
  int32_t* status;
};

// Workgroups of the attention kernel, one per compute unit of an MI355X, and
// the fewest cache rows a workgroup takes (a call with fewer rows to read
// uses fewer workgroups: each costs its share of the join).  In tiles that is 1 of
// units of 32, 2 of 64, 4 of 128.  Measured for one request, us a call with 64 /
// 128 / 256 rows: a token of 16 heads over 1,000 rows 21.1 / 21.1 / 23.8 (64 and
// 128 are a tile both), over 8,000 27.9 / 27.9 / 23.7; of 64 heads over 1,000 21.4
// / 21.2 / 25.6, over 4,000 28.5 / 26.1 / 29.1, over 30,000 61.8 / 61.9 / 47.3 (the
// join reads a part of every workgroup); 8 drafts of 16 heads over 2,000 29.1 /
// 29.1 / 33.4, 64 drafts over 1,000 35.9 / 40.0 / 40.5.
constexpr int kAttendWorkgroups = 256;
constexpr int kAttendLeastRows = 128;

// A unit's begin and end (its queries in, its outputs out), as the rows that
// take the same time.  Measured on 16 prompts of some 2,000 tokens with 32
// heads: 192 rows 1.66 ms, 256 1.51, 320 1.485, 384 1.53, 480 1.59.
constexpr int kAttendUnitRows = 320;

// Most units of a call whose workgroups plan for themselves, four per lane:
// 1 unit 21.1 us in all against 26.0 with the plan's own launch, 64 units 123.3
// against 128.5, 128 units 129 against 132.5.  (The plan kernel's cut units, at
// most one per boundary between workgroups, share the table.)
constexpr int kAttendPlanUnits = 256;
static_assert(kAttendPlanUnits >= kAttendWorkgroups - 1, "places for every cut unit");

struct AttendHead {            // written by the plan
  int32_t nsplit;              // units cut between workgroups
  int32_t pad[3];
};
struct AttendStart {           // where a workgroup begins, and the one before it ends (slot S: the end)
  int32_t slot, unit, tile, pad;
};
struct AttendSplit {           // a unit and its parts, which lie with workgroups wg0 ..
  int32_t slot, unit, wg0, parts;
};

struct AttendParams {
  CacheView cache;
  int32_t ratio;
  int32_t heads;
  DivMagic head_div;           // division by heads
  int32_t num_slots;
  int32_t draft_len;           // tokens per slot (offsets NULL)
  const uint16_t* q;
  int64_t q_stride;            // elements between tokens
  int64_t q_hstride;           // elements between heads
  int64_t q_rows;              // token rows q, out and lse hold
  const int32_t* offsets;      // packed tokens, or NULL
  const int32_t* start_pos;
  const int32_t* page_table;
  int64_t pt_stride;
  int64_t pt_width;
  const uint64_t* tree;        // ancestor masks, or NULL
  float scale_log2;            // scale * log2(e)
  const float* sink;           // nullable
  uint16_t* out;
  int64_t out_stride;
  int64_t out_hstride;
  float* lse;                  // nullable
  int32_t* status;
  int64_t units_max;           // units the call can have at the most
  int32_t plan_units;          // > 0: most units of a slot, and every workgroup plans for itself
  DivMagic plan_div;           // division by plan_units
  // workspace
  AttendHead* head;
  AttendStart* starts;         // [kAttendWorkgroups + 1]
  AttendSplit* splits;         // [kAttendPlanUnits]
  float4* part_ml;             // [2 * kAttendWorkgroups][queries of a unit]: max, sum, rounded sum
  float* part_o;               // the same, 512 dims each
};

// The launchers, as those of launch.hpp (several kernels in a row).  Weak: a
// host-only build of the C ABI may leave them out, and the calls that need
// them then report that nothing can be launched.
__attribute__((weak)) hipError_t launch_slot_map(const SlotMapParams& p, hipStream_t stream);
// qblocks: 32-query blocks per unit (1, 2 or 4)
__attribute__((weak)) hipError_t launch_attend(const AttendParams& p, int qblocks, hipStream_t stream);

}  // namespace kvc
