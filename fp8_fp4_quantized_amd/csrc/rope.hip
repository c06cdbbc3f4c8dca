// rope.hip -- the rotary table, scaled for long contexts or not, and the
// rotation of query heads and attention outputs by it (gfx950).
//
// Table: freqs[i][2j], freqs[i][2j + 1] = mscale * (cos, sin) of the angle
// (first + i) * w_j.  The speeds w_j come from the host in 64 bits as half turns
// a position; a thread makes its first entry and the turn from one of its
// entries to the next by sincospi in 64 bits and goes on by complex products in
// 64 bits (kTableRun of them: the error stays below 2^-45, far under the one
// rounding to fp32).  Bound by the writes.
//
// Rotation: with (c, s) = freqs[position] the pair (a, b) becomes
//   (a c - b s, a s + b c), transposed (a c + b s, b c - a s),
// in fp32, rounded once to the heads' type.  Bound by HBM; in place only the
// rotated dims move.
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
// dims, strides and addresses that the kernel by 16 bytes does not take.
template <int T>
__global__ __launch_bounds__(kRopeBlock) void rope_elements_kernel(RopeRowsParams p) {
  typedef typename Elem<T>::type E;
  const int64_t u0 = (int64_t)blockIdx.x * kRopeBlock;
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

hipError_t launch_elements(RopeRowsParams p, hipStream_t stream) {
  p.head_units = p.rot / 2 + (p.in_place ? 0 : p.dim - p.rot);
  p.token_units = p.head_units * p.heads;
  p.head_div = div_magic((uint32_t)p.head_units);
  p.token_div = div_magic((uint32_t)p.token_units);
  p.units = p.tokens * p.token_units;
  const dim3 grid((uint32_t)((p.units + kRopeBlock - 1) / kRopeBlock));
  switch (p.type) {
    case kRopeBf16: rope_elements_kernel<kRopeBf16><<<grid, kRopeBlock, 0, stream>>>(p); break;
    case kRopeF16: rope_elements_kernel<kRopeF16><<<grid, kRopeBlock, 0, stream>>>(p); break;
    default: rope_elements_kernel<kRopeF32><<<grid, kRopeBlock, 0, stream>>>(p); break;
  }
  return hipGetLastError();
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

hipError_t launch_rope_rows(const RopeRowsParams& p, hipStream_t stream) { return launch_elements(p, stream); }

}  // namespace kvc
