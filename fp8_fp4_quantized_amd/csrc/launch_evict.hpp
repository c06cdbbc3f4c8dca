// launch_evict.hpp -- arguments and launchers of the rotary table and rotation,
// and of the eviction: attention weights of cached rows, the choice of the rows
// kept, their move to other pages.
#pragma once

#include "launch_attend.hpp"

namespace kvc {

// ---------------------------------------------------------------- rotary
constexpr int kRopeMaxPairs = 256;

struct RopeTableParams {
  float* freqs;                // [n, 2 * pairs]
  int64_t n;
  int64_t first;               // position of the first row
  int32_t pairs;
  double mscale;
  double speed[kRopeMaxPairs]; // w_j / pi: half turns a position
};

enum RopeType : int32_t { kRopeBf16 = 0, kRopeF16 = 1, kRopeF32 = 2 };

struct RopeRowsParams {
  const void* x;
  int64_t x_stride, x_hstride;       // elements between tokens, heads
  void* out;
  int64_t out_stride, out_hstride;
  int64_t tokens;
  int32_t heads, dim, rot, offset;
  int32_t type;                // RopeType
  int32_t half;                // pairs (j, j + rot / 2); else (2j, 2j + 1)
  int32_t transpose;
  int32_t in_place;            // out is x: only the rotated dims are written
  const int32_t* positions;
  const float* freqs;          // [max_pos, rot]
  int64_t max_pos;
  int32_t* status;
  // set by the launcher: units of a head, of a token, and the division by them
  int64_t units;
  int32_t head_units, token_units;
  DivMagic head_div, token_div;
};

// ---------------------------------------------------------------- weights
// Workgroups of the kernel for many queries, one per compute unit
constexpr int kWeighWorkgroups = 256;
constexpr int kWeighRows = 256;       // rows of a block of it: 4 waves of 64

// Places for the sums of slots that are cut into segments (256 floats each)
constexpr int kWeighParts = 16384;

struct WeighHead {             // written by the kernel, for the one that joins its sums
  int32_t cut;                 // segments of 2^cut tokens
  int32_t pad[63];
};

struct WeighParams {
  CacheView cache;
  int32_t ratio;
  int32_t heads;
  DivMagic head_div;
  int32_t num_slots;
  int32_t draft_len;           // tokens per slot (offsets NULL)
  const uint16_t* q;
  int64_t q_stride, q_hstride; // elements
  int64_t q_rows;
  const float* lse;            // [q_rows, heads]
  const int32_t* offsets;      // packed tokens, or NULL
  const int32_t* start_pos;
  const int32_t* page_table;
  int64_t pt_stride, pt_width;
  const uint64_t* tree;        // nullable
  float scale_log2;
  float decay;
  const float* prev;           // nullable; may be weights
  int64_t prev_stride;
  float* weights;
  int64_t w_stride, w_width;
  int32_t* status;
  // workspace of the kernel for many queries
  WeighHead* head;
  float* parts;                // [kWeighParts][kWeighRows]
};

// ---------------------------------------------------------------- choice
// Rows of weights that one workgroup keeps in registers; of longer ones of up to
// kSelectSegmentSlots slots, a slot's rows are cut into segments of at least
// kSelectSegmentRows, kSelectSegments for all slots together at the most; those of
// more slots are read by one workgroup a slot, once a digit.  Measured, us a call:
// in registers and in segments, 64 slots of 16,384 rows 13 and 26, of 17,000 17 and 27, of
// 32,768 26 and 29 (512 slots: 57, and 73 read once a digit); in segments and read once a
// digit, 40,000 rows of 64 slots 29 and 47, of 128 slots 50 and 55, of 200 slots 69 and 69,
// 100,000 of 64 slots 51 and 129.  Segments of 8,192 rows take a million rows of one slot
// from 34 to 36.  The width alone decides: 64 slots of 4,200 to 16,384 rows take 12 in rows
// of weights that wide, 20 in 32,768 and 47 in 131,072 or more; 200 slots 12, 21 and 22.
constexpr int kSelectRegisterRows = 32768;
constexpr int kSelectSegmentSlots = 128;
constexpr int kSelectSegmentRows = 16384;
constexpr int kSelectSegments = 512;
// words of a segment in the workspace: three histograms with their sums, a state of 4
constexpr int kSelectWords = 2048 + 64;

struct SelectParams {
  int32_t ratio;
  int32_t num_slots;
  const int32_t* lens;
  const float* weights;
  int64_t w_stride, w_width;
  int32_t budget;
  const int32_t* budgets;      // nullable
  int32_t first, recent;
  int32_t* kept;
  int64_t kept_stride;
  int32_t kept_width;
  int32_t* counts;
  float* kept_weights;         // nullable
  int64_t kw_stride;
  int32_t* status;
  // segments a slot (0: none), their rows, and the workspace
  int32_t segments;
  int64_t segment_rows;
  uint32_t* hists;             // [3][slots][segments][kSelectWords]
  int32_t* states;             // [slots][segments][4]
};

// ---------------------------------------------------------------- move
struct CompactParams {
  CacheView cache;
  int32_t ratio;
  int32_t num_slots;
  const int32_t* lens;
  const int32_t* kept;
  int64_t kept_stride;
  int32_t kept_width;
  const int32_t* counts;
  const int32_t* page_table;
  int64_t pt_stride, pt_width;
  const int32_t* free_pages;
  int64_t n_free;
  int32_t* new_table;
  int64_t nt_stride;
  int32_t* new_lens;
  const float* kept_weights;   // nullable, with weights
  int64_t kw_stride;
  float* weights;
  int64_t w_stride, w_width;
  int32_t* freed;              // nullable
  int64_t freed_cap;
  int32_t* totals;             // nullable
  int32_t* status;
};

// Launchers, weak like those of launch_attend.hpp
__attribute__((weak)) hipError_t launch_rope_table(const RopeTableParams& p, hipStream_t stream);
__attribute__((weak)) hipError_t launch_rope_rows(const RopeRowsParams& p, hipStream_t stream);
// few: the queries of a slot fit the kernel that keeps them (kWeighFew at the most)
constexpr int kWeighFew = 128;
__attribute__((weak)) hipError_t launch_weigh(const WeighParams& p, int64_t slot_queries, hipStream_t stream);
__attribute__((weak)) hipError_t launch_select(const SelectParams& p, hipStream_t stream);
__attribute__((weak)) hipError_t launch_compact(const CompactParams& p, hipStream_t stream);

}  // namespace kvc
