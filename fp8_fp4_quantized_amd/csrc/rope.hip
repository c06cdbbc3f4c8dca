// rope.hip -- the rotary table, scaled for long contexts or not, and the
// rotation of query heads and attention outputs by it (gfx950).
//
// Table: freqs[i][2j], freqs[i][2j + 1] = mscale * (cos, sin) of the angle
// (first + i) * w_j.  The speeds w_j come from the host in 64 bits as half turns
// a position; a thread makes its first entry and the turn from one of its
// entries to the next by sincospi in 64 bits and goes on by complex products in
// 64 bits, kTableRun of them.  Where the positions of a turn are a power of two their
// angle is exact and the products add 2^-48; elsewhere (10 dims: 51 positions) the
// angle, up to 27 half turns at speeds up to 1, is rounded, which 31 products carry to
// 31 pi 2^-49, below 2^-42, and in proportion for faster speeds: far under the one rounding
// to fp32.  The angle of the first entry has a rounding of its own size.  Bound by the
// writes: a million positions of 64 dims, 268 MB, take 46 to 48 us (5.6 to 5.8 TB/s);
// 4,096 of them 4.6.
//
// Rotation: with (c, s) = freqs[position] the pair (a, b) becomes
//   (a c - b s, a s + b c), transposed (a c + b s, b c - a s),
// in fp32, rounded once to the heads' type.  Bound by HBM; in place only the
// rotated dims move.  A decode step's 64 tokens of 64 heads take 4 us.
#include <algorithm>
#include <type_traits>

#include "launch_evict.hpp"
#include "layout.hpp"
#include "row_ops.hpp"

namespace kvc {

namespace {

constexpr int kRopeBlock = 256;

// ------------------------------------------------------------------ table
constexpr int kTableRun = 32;

// V pairs a thread (2 where their number is even: 16-byte stores)
template <int V>
__global__ __launch_bounds__(kRopeBlock) void rope_table_kernel(RopeTableParams p) {
  const int groups = p.pairs / V;             // threads of a position, 1 .. kRopeBlock
  const int rows = kRopeBlock / groups;       // positions a turn of the workgroup
  const int r = (int)threadIdx.x / groups, g = (int)threadIdx.x - r * groups;
  if (r >= rows) return;
  const int64_t i0 = (int64_t)blockIdx.x * rows * kTableRun + r;
  if (i0 >= p.n) return;
  double c[V], s[V], tc[V], ts[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const double w = p.speed[g * V + v];
    sincospi((double)(p.first + i0) * w, &s[v], &c[v]);
    sincospi((double)rows * w, &ts[v], &tc[v]);
    c[v] *= p.mscale;
    s[v] *= p.mscale;
  }
  float* at = p.freqs + (i0 * p.pairs + g * V) * 2;
  for (int k = 0; k < kTableRun; ++k) {
    const int64_t i = i0 + (int64_t)k * rows;
    if (i >= p.n) break;
    if constexpr (V == 2) {
      typedef float f32x4v __attribute__((ext_vector_type(4)));
      *(f32x4v*)at = f32x4v{(float)c[0], (float)s[0], (float)c[1], (float)s[1]};
    } else {
      *(f32x2*)at = f32x2{(float)c[0], (float)s[0]};
    }
    at += (int64_t)rows * p.pairs * 2;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const double nc = __builtin_fma(c[v], tc[v], -(s[v] * ts[v]));
      s[v] = __builtin_fma(s[v], tc[v], c[v] * ts[v]);
      c[v] = nc;
    }
  }
}

// ------------------------------------------------------------------ rotation
template <int T> struct Elem;
template <> struct Elem<kRopeBf16> {
  typedef uint16_t type;
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t put(float v) { return (uint16_t)pack_bf16(v, 0.0f); }
};
template <> struct Elem<kRopeF16> {
  typedef uint16_t type;
  static __device__ __forceinline__ float get(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t put(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
template <> struct Elem<kRopeF32> {
  typedef float type;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

struct Turned {
  float a, b;
};
__device__ __forceinline__ Turned turn(float a, float b, float c, float s) {
  return Turned{__builtin_fmaf(a, c, -(b * s)), __builtin_fmaf(a, s, b * c)};
}

// a unit's place: its token, head and unit of the head
struct Unit {
  int64_t token;
  int32_t head, k;
};
__device__ __forceinline__ Unit unit_at(const RopeRowsParams& p, int64_t token0, uint32_t rem) {
  const uint32_t t = udiv_magic(rem, p.token_div.m, p.token_div.sh1, p.token_div.sh2);
  rem -= t * (uint32_t)p.token_units;
  const uint32_t h = udiv_magic(rem, p.head_div.m, p.head_div.sh1, p.head_div.sh2);
  return Unit{token0 + t, (int32_t)h, (int32_t)(rem - h * (uint32_t)p.head_units)};
}

// whether the token's position is one of the table; flags one that is not
__device__ __forceinline__ bool position_ok(const RopeRowsParams& p, int32_t pos) {
  if (pos >= 0 && pos < p.max_pos) return true;
  if (p.status != nullptr) atomicOr(p.status, kStPosRange);
  return false;
}

// Element by element: a unit is one pair, or one dim that is only copied.  For
// dims, strides and addresses that the kernel by 16 bytes does not take.  u0: the
// workgroup's first unit.
template <int T>
__device__ __forceinline__ void rope_element(const RopeRowsParams& p, int64_t u0) {
  typedef typename Elem<T>::type E;
  const int64_t token0 = u0 / p.token_units;
  if (u0 + threadIdx.x >= p.units) return;
  const Unit u = unit_at(p, token0, (uint32_t)(u0 - token0 * p.token_units) + threadIdx.x);
  const int32_t pos = p.positions[u.token];
  if (!position_ok(p, pos)) return;
  const E* x = (const E*)p.x + u.token * p.x_stride + u.head * p.x_hstride;
  E* out = (E*)p.out + u.token * p.out_stride + u.head * p.out_hstride;
  const int pairs = p.rot / 2;
  if (u.k < pairs) {
    const int da = p.offset + (p.half ? u.k : 2 * u.k), db = da + (p.half ? pairs : 1);
    const float c = p.freqs[(int64_t)pos * p.rot + 2 * u.k];
    float s = p.freqs[(int64_t)pos * p.rot + 2 * u.k + 1];
    if (p.transpose) s = -s;
    const Turned r = turn(Elem<T>::get(x[da]), Elem<T>::get(x[db]), c, s);
    out[da] = Elem<T>::put(r.a);
    out[db] = Elem<T>::put(r.b);
  } else {
    const int d = u.k - pairs;                // of the dims that are not rotated
    const int at = d < p.offset ? d : d + p.rot;
    out[at] = x[at];
  }
}

// (a launch has less than 2^32 threads, and 20 GB of heads have as many units)
constexpr int64_t kElementsGrid = int64_t(1) << 23;

template <int T>
__global__ __launch_bounds__(kRopeBlock) void rope_elements_kernel(RopeRowsParams p) {
  for (int64_t u0 = (int64_t)blockIdx.x * kRopeBlock; u0 < p.units; u0 += (int64_t)gridDim.x * kRopeBlock)
    rope_element<T>(p, u0);
}

hipError_t launch_elements(RopeRowsParams p, hipStream_t stream) {
  p.head_units = p.rot / 2 + (p.in_place ? 0 : p.dim - p.rot);
  p.token_units = p.head_units * p.heads;
  p.head_div = div_magic((uint32_t)p.head_units);
  p.token_div = div_magic((uint32_t)p.token_units);
  p.units = p.tokens * p.token_units;
  const dim3 grid((uint32_t)std::min((p.units + kRopeBlock - 1) / kRopeBlock, kElementsGrid));
  switch (p.type) {
    case kRopeBf16: rope_elements_kernel<kRopeBf16><<<grid, kRopeBlock, 0, stream>>>(p); break;
    case kRopeF16: rope_elements_kernel<kRopeF16><<<grid, kRopeBlock, 0, stream>>>(p); break;
    default: rope_elements_kernel<kRopeF32><<<grid, kRopeBlock, 0, stream>>>(p); break;
  }
  return hipGetLastError();
}

// By 16 bytes, E dims: a unit is 16 bytes of a head -- with pairs of halves, the
// 16 bytes of either half that belong together.  A thread takes kUnits of them, all
// loads issued before the first store.
constexpr int kUnits = 4;

template <int T>
struct Vec {
  static constexpr int E = T == kRopeF32 ? 4 : 8;
  float f[E];
  __device__ __forceinline__ explicit Vec(u32x4 v) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (T == kRopeF32) f[e] = __uint_as_float(v[e]);
      else f[e] = Elem<T>::get((uint16_t)(v[e / 2] >> (16 * (e & 1))));
    }
  }
  __device__ __forceinline__ u32x4 bits() const {
    u32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (T == kRopeF32) v[k] = __float_as_uint(f[k]);
      else if constexpr (T == kRopeBf16) v[k] = pack_bf16(f[2 * k], f[2 * k + 1]);
      else v[k] = (uint32_t)Elem<T>::put(f[2 * k]) | (uint32_t)Elem<T>::put(f[2 * k + 1]) << 16;
    }
    return v;
  }
};

// (a table's rows begin at multiples of 8 bytes)
typedef float f32x4_8 __attribute__((ext_vector_type(4), aligned(8)));

template <int T, bool HALF>
__global__ __launch_bounds__(kRopeBlock) void rope_vectors_kernel(RopeRowsParams p) {
  constexpr int E = Vec<T>::E, size = 16 / E;
  const int64_t u0 = (int64_t)blockIdx.x * (kRopeBlock * kUnits);
  const int64_t token0 = u0 / p.token_units;
  const uint32_t rem0 = (uint32_t)(u0 - token0 * p.token_units) + threadIdx.x;
  const int pair_units = HALF ? p.rot / 2 / E : 0;
  u32x4 a[kUnits], b[kUnits];
  uint8_t* out[kUnits];
  int32_t pos[kUnits], d[kUnits];             // d: first dim of the unit (of its half)
  bool pair[kUnits];                          // HALF: a unit of two
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    out[i] = nullptr;
    if (u0 + i * kRopeBlock + threadIdx.x >= p.units) continue;
    const Unit u = unit_at(p, token0, rem0 + i * kRopeBlock);
    pos[i] = p.positions[u.token];
    pair[i] = HALF && u.k < pair_units;
    if constexpr (HALF) {
      const int c = (u.k - pair_units) * E;   // dims that are copied
      d[i] = pair[i] ? p.offset + u.k * E : c < p.offset ? c : c + p.rot;
    } else {
      d[i] = ((p.in_place ? p.offset / E : 0) + u.k) * E;
    }
    const uint8_t* x = (const uint8_t*)p.x + (u.token * p.x_stride + u.head * p.x_hstride + d[i]) * size;
    out[i] = (uint8_t*)p.out + (u.token * p.out_stride + u.head * p.out_hstride + d[i]) * size;
    a[i] = *(const u32x4*)x;
    if (HALF && pair[i]) b[i] = *(const u32x4*)(x + p.rot / 2 * size);
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (out[i] == nullptr || !position_ok(p, pos[i])) continue;
    const float* f = p.freqs + (int64_t)pos[i] * p.rot;
    if constexpr (HALF) {
      if (pair[i]) {
        Vec<T> va(a[i]), vb(b[i]);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const f32x4_8 t = *(const f32x4_8*)(f + 2 * (d[i] - p.offset + e));
          const Turned r0 = turn(va.f[e], vb.f[e], t[0], p.transpose ? -t[1] : t[1]);
          const Turned r1 = turn(va.f[e + 1], vb.f[e + 1], t[2], p.transpose ? -t[3] : t[3]);
          va.f[e] = r0.a, vb.f[e] = r0.b, va.f[e + 1] = r1.a, vb.f[e + 1] = r1.b;
        }
        a[i] = va.bits();
        *(u32x4*)(out[i] + p.rot / 2 * size) = vb.bits();
      }
    } else {
      const int at = d[i] - p.offset;         // (even)
      if (at >= 0 && at + E <= p.rot) {
        Vec<T> v(a[i]);
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const f32x4_8 t = *(const f32x4_8*)(f + at + e);
          const Turned r0 = turn(v.f[e], v.f[e + 1], t[0], p.transpose ? -t[1] : t[1]);
          const Turned r1 = turn(v.f[e + 2], v.f[e + 3], t[2], p.transpose ? -t[3] : t[3]);
          v.f[e] = r0.a, v.f[e + 1] = r0.b, v.f[e + 2] = r1.a, v.f[e + 3] = r1.b;
        }
        a[i] = v.bits();
      } else if (at + E > 0 && at < p.rot) {
        // the rotated dims begin or end in the unit
        Vec<T> v(a[i]);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          if (at + e < 0 || at + e >= p.rot) continue;
          const f32x2 t = *(const f32x2*)(f + at + e);
          const Turned r = turn(v.f[e], v.f[e + 1], t[0], p.transpose ? -t[1] : t[1]);
          v.f[e] = r.a, v.f[e + 1] = r.b;
        }
        // (dims that are copied keep their bits: a conversion changes some NaNs'.  In
        // place they are not stored at all: another stream may be writing them.  A 4-byte
        // word is rotated whole or not, the first dim being even)
        const u32x4 made = v.bits();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = at + k * E / 4;
          const bool turned = r >= 0 && r < p.rot;
          if (p.in_place && turned) ((uint32_t*)out[i])[k] = made[k];
          a[i][k] = turned ? made[k] : a[i][k];
        }
        if (p.in_place) continue;
      }
    }
    *(u32x4*)out[i] = a[i];
  }
}

// 16 bytes at an address of any element
typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));

// The same for any offset, dims, strides and addresses, into another place than
// x: every unit makes its own E dims (the last unit of a head ends with it and may
// overlap the one before, which writes the same), whose partners it has, or
// fetches one by one.  Addresses need not be multiples of 16: loads and stores of
// 16 bytes take any.
template <int T>
__global__ __launch_bounds__(kRopeBlock) void rope_any_kernel(RopeRowsParams p) {
  typedef typename Elem<T>::type Ty;
  typedef typename std::conditional<T == kRopeF32, u32x4_4, u32x4_2>::type u32x4_any;
  constexpr int E = Vec<T>::E;
  const int64_t u0 = (int64_t)blockIdx.x * (kRopeBlock * kUnits);
  const int64_t token0 = u0 / p.token_units;
  const uint32_t rem0 = (uint32_t)(u0 - token0 * p.token_units) + threadIdx.x;
  const int apart = p.rot / 2;
  u32x4 v[kUnits];
  const Ty* x[kUnits];
  Ty* out[kUnits];
  int32_t pos[kUnits], rel[kUnits];           // rel: first dim of the unit from the first rotated one
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    out[i] = nullptr;
    if (u0 + i * kRopeBlock + threadIdx.x >= p.units) continue;
    const Unit u = unit_at(p, token0, rem0 + i * kRopeBlock);
    pos[i] = p.positions[u.token];
    const int d = min(u.k * E, p.dim - E);
    rel[i] = d - p.offset;
    x[i] = (const Ty*)p.x + u.token * p.x_stride + u.head * p.x_hstride + d;
    out[i] = (Ty*)p.out + u.token * p.out_stride + u.head * p.out_hstride + d;
    v[i] = *(const u32x4_any*)x[i];
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (out[i] == nullptr || !position_ok(p, pos[i])) continue;
    if (rel[i] + E > 0 && rel[i] < p.rot) {
      const f32x2* f = (const f32x2*)(p.freqs + (int64_t)pos[i] * p.rot);
      const Vec<T> own(v[i]);
      Vec<T> made = own;
      // partners: in the unit but for one at either end, or half the rotated dims away
      float other[E];
      if (!p.half) {
#pragma unroll
        for (int e = 0; e < E; ++e) other[e] = ((rel[i] + e) & 1) != 0 ? own.f[max(e - 1, 0)] : own.f[min(e + 1, E - 1)];
        if ((rel[i] & 1) != 0) {
          if (rel[i] > 0) other[0] = Elem<T>::get(x[i][-1]);
          if (rel[i] + E < p.rot) other[E - 1] = Elem<T>::get(x[i][E]);
        }
      } else if (rel[i] >= 0 && rel[i] + E <= apart) {
        const Vec<T> w(*(const u32x4_any*)(x[i] + apart));
#pragma unroll
        for (int e = 0; e < E; ++e) other[e] = w.f[e];
      } else if (rel[i] >= apart && rel[i] + E <= p.rot) {
        const Vec<T> w(*(const u32x4_any*)(x[i] - apart));
#pragma unroll
        for (int e = 0; e < E; ++e) other[e] = w.f[e];
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int r = rel[i] + e;
          other[e] = r >= 0 && r < p.rot ? Elem<T>::get(x[i][r < apart ? e + apart : e - apart]) : 0.0f;
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int r = min(max(rel[i] + e, 0), p.rot - 1);
        const bool second = p.half ? r >= apart : (r & 1) != 0;
        const f32x2 t = f[p.half ? (second ? r - apart : r) : r >> 1];
        const float sn = p.transpose ? -t[1] : t[1];
        const float y = second ? turn(other[e], own.f[e], t[0], sn).b : turn(own.f[e], other[e], t[0], sn).a;
        if (r == rel[i] + e) made.f[e] = y;
      }
      // (dims that are copied keep their bits: a conversion changes some NaNs')
      constexpr int per = E / 4;
      const u32x4 bits = made.bits();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t turned = 0;
#pragma unroll
        for (int e = 0; e < per; ++e) {
          const int r = rel[i] + k * per + e;
          if (r >= 0 && r < p.rot) turned |= (per == 1 ? 0xFFFFFFFFu : 0xFFFFu) << (16 * e);
        }
        v[i][k] = (bits[k] & turned) | (v[i][k] & ~turned);
      }
    }
    *(u32x4_any*)out[i] = v[i];
  }
}

template <int T>
hipError_t launch_any(RopeRowsParams p, hipStream_t stream) {
  constexpr int E = Vec<T>::E;
  p.head_units = (p.dim + E - 1) / E;
  p.token_units = p.head_units * p.heads;
  p.head_div = div_magic((uint32_t)p.head_units);
  p.token_div = div_magic((uint32_t)p.token_units);
  p.units = p.tokens * p.token_units;
  const dim3 grid((uint32_t)((p.units + kRopeBlock * kUnits - 1) / (kRopeBlock * kUnits)));
  rope_any_kernel<T><<<grid, kRopeBlock, 0, stream>>>(p);
  return hipGetLastError();
}

template <int T>
hipError_t launch_vectors(RopeRowsParams p, hipStream_t stream) {
  constexpr int E = Vec<T>::E;
  if (p.half) p.head_units = p.rot / 2 / E + (p.in_place ? 0 : (p.dim - p.rot) / E);
  else if (p.in_place) p.head_units = (p.offset + p.rot + E - 1) / E - p.offset / E;
  else p.head_units = p.dim / E;
  p.token_units = p.head_units * p.heads;
  p.head_div = div_magic((uint32_t)p.head_units);
  p.token_div = div_magic((uint32_t)p.token_units);
  p.units = p.tokens * p.token_units;
  const dim3 grid((uint32_t)((p.units + kRopeBlock * kUnits - 1) / (kRopeBlock * kUnits)));
  if (p.half) rope_vectors_kernel<T, true><<<grid, kRopeBlock, 0, stream>>>(p);
  else rope_vectors_kernel<T, false><<<grid, kRopeBlock, 0, stream>>>(p);
  return hipGetLastError();
}

// Measured, 8,192 tokens of 128 heads of 512 dims in bf16 from one tensor to another,
// 2.15 GB: 366 us with pairs of neighbours and 414 with pairs of halves (5.9 and 5.2 TB/s);
// by rope_any_kernel 565 and 686, which also takes an odd offset (665) and 511 dims
// (734); element by element 1,745.  fp16 takes the same, fp32 370 and 389 for as many bytes.
// In place all dims 386, the last 64 48, 36 dims from 6 on (half of 16 bytes at the ends,
// stored by words) 55; pair by pair, an odd offset, 1,275.
// Whether heads can be taken by 16 bytes: addresses, strides and dims of whole
// ones, pairs inside one of them (or their halves at whole ones).
bool by_vectors(const RopeRowsParams& p) {
  const int E = p.type == kRopeF32 ? 4 : 8;
  const int64_t strides = p.x_stride | p.x_hstride | p.out_stride | p.out_hstride | p.dim;
  if (strides % E != 0 || (((uintptr_t)p.x | (uintptr_t)p.out) & 15u) != 0) return false;
  return p.half ? p.offset % E == 0 && p.rot / 2 % E == 0 : p.offset % 2 == 0;
}

}  // namespace

hipError_t launch_rope_table(const RopeTableParams& p, hipStream_t stream) {
  const bool two = p.pairs % 2 == 0;
  const int rows = kRopeBlock / (two ? p.pairs / 2 : p.pairs);
  const dim3 grid((uint32_t)((p.n + (int64_t)rows * kTableRun - 1) / ((int64_t)rows * kTableRun)));
  if (two) rope_table_kernel<2><<<grid, kRopeBlock, 0, stream>>>(p);
  else rope_table_kernel<1><<<grid, kRopeBlock, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_rope_rows(const RopeRowsParams& p, hipStream_t stream) {
  if (!by_vectors(p)) {
    // in place a unit's partners would be another's to write
    if (p.in_place || p.dim < (p.type == kRopeF32 ? 4 : 8)) return launch_elements(p, stream);
    switch (p.type) {
      case kRopeBf16: return launch_any<kRopeBf16>(p, stream);
      case kRopeF16: return launch_any<kRopeF16>(p, stream);
      default: return launch_any<kRopeF32>(p, stream);
    }
  }
  switch (p.type) {
    case kRopeBf16: return launch_vectors<kRopeBf16>(p, stream);
    case kRopeF16: return launch_vectors<kRopeF16>(p, stream);
    default: return launch_vectors<kRopeF32>(p, stream);
  }
}

}  // namespace kvc
