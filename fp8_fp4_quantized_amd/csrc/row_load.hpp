// row_load.hpp -- one cached row on one wavefront: the lanes' loads of its
// codes and scales, and their expansion to bf16 (8 dims per lane).
#pragma once

#include "row_ops.hpp"

namespace kvc {

template <int L> struct LaneCodes;          // this lane's share of a row
template <> struct LaneCodes<kV41> { uint2 codes; uint32_t scale; };
template <> struct LaneCodes<kV41Fp4> { uint32_t codes; uint32_t scale; };
template <> struct LaneCodes<kV4> { uint4 raw; uint32_t scale; };

// Loads from the row's own base (the slot is the same on every lane).  A
// row's scale part shares its cache line with the scale parts of the page's
// other rows, so it is always a cached load (non-temporal: 6% slower on a
// 262,144-id gather); the codes take CPOL.
template <int L, int CPOL>
__device__ __forceinline__ LaneCodes<L> load_lane(const PagedKV<L>& kv, int64_t slot, int lane) {
  LaneCodes<L> r;
  if constexpr (L == kV41) {
    r.codes = ld_u2_buf<CPOL>(kv.data(slot), 8u * lane);
    r.scale = ld_u8_dev(kv.scale(slot), (uint32_t)lane >> 2);
  } else if constexpr (L == kV41Fp4) {
    r.codes = ld_u32_buf<CPOL>(kv.data(slot), 4u * lane);
    r.scale = ld_u8_dev(kv.scale(slot), (uint32_t)lane >> 1);
  } else {
    const uint8_t* d = kv.data(slot);
    if (lane < kRopeLane0) {
      const uint2 c = ld_u2_buf<CPOL>(d, 8u * lane);
      r.raw = make_uint4(c.x, c.y, 0u, 0u);
      r.scale = ld_u8_dev(kv.scale(slot), (uint32_t)lane >> 3);
    } else {
      r.raw = ld_u4_buf<CPOL>(d, kNope + 16u * (lane - kRopeLane0));
      r.scale = 0;
    }
  }
  return r;
}

template <int L>
__device__ __forceinline__ uint4 decode_lane(const LaneCodes<L>& c, int lane);
template <>
__device__ __forceinline__ uint4 decode_lane<kV41>(const LaneCodes<kV41>& c, int) {
  return dq_fp8x8(c.codes, c.scale);
}
template <>
__device__ __forceinline__ uint4 decode_lane<kV41Fp4>(const LaneCodes<kV41Fp4>& c, int) {
  return dq_fp4x8(c.codes, c.scale);
}
template <>
__device__ __forceinline__ uint4 decode_lane<kV4>(const LaneCodes<kV4>& c, int lane) {
  if (lane >= kRopeLane0) return c.raw;
  return dq_fp8x8(make_uint2(c.raw.x, c.raw.y), c.scale);
}

}  // namespace kvc
