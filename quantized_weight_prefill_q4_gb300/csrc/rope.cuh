// Rotations by position (include/apr_rope.h) as the kernels see them.
//
// A head is cut into units of eight dims, one for each lane of a group of lanes: the
// units below rot / 8 are four pairs (dims 4 u .. and rot / 2 + 4 u .., or 8 u .. in
// the interleaved order), the others eight dims that pass. A lane keeps its unit over
// rows and heads, so which table columns, axes and norm weights are its own is settled once.
#pragma once

#include "kv8.cuh"

namespace apr {

struct RopeView {
  const float2* table;
  const uint8_t* axis;    // nullptr: axis 0
  const int* positions;   // nullptr: the row's position in its sequence
  long long positions_ld;
  unsigned* status;
  int num_positions, pairs, num_axes, interleaved;
};

// The norm of the heads, and rows into rows.
struct RopeRows {
  const void* x;
  void* out;
  long long ldx, ldo;
  const float* norm;  // nullptr: none
  float eps;
  int num_rows, heads, dim;
  int heads_a_group;  // that a group of lanes does of one row
};

// Unit u of a head: dims d0 .. d0 + 3 and d1 .. d1 + 3.
struct RopeUnit {
  int d0, d1, pair;  // its first pair; -1: the dims pass
  uint32_t axes;     // of its four pairs, a byte each
};
__device__ __forceinline__ RopeUnit rope_unit(const RopeView& r, int u) {
  const bool turned = 4 * u < r.pairs;
  RopeUnit w;
  w.pair = turned ? 4 * u : -1;
  w.d0 = turned && !r.interleaved ? 4 * u : 8 * u;
  w.d1 = turned && !r.interleaved ? r.pairs + 4 * u : 8 * u + 4;
  w.axes = turned && r.axis ? *reinterpret_cast<const uint32_t*>(r.axis + 4 * u) : 0;
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    if ((int)(w.axes >> i & 255) >= r.num_axes) {
      atomicOr(r.status, kStatusBadIndex);
      w.axes &= ~(255u << i);
    }
  return w;
}

// The cosines and sines of a unit's pairs for packed row `row`, whose position in
// its sequence is `own` (what counts where no positions are given).
struct RopeTurn {
  float2 t[4];
};
// (`bad` where the table does not have the position: told at once, so that no load waits for a report.)
__device__ __forceinline__ int rope_position(const RopeView& r, int axis, int row, int own, bool& bad) {
  const int p = r.positions ? r.positions[axis * r.positions_ld + row] : max(own, 0);
  const bool here = (unsigned)p < (unsigned)r.num_positions;
  bad |= !here;
  return here ? p : 0;
}
__device__ __forceinline__ RopeTurn rope_turn(const RopeView& r, const RopeUnit& u, int row, int own) {
  RopeTurn w;
  if (u.pair < 0) return w;
  const int a = (int)(u.axes & 255);
  bool bad = false;
  const float2* at = r.table + (size_t)rope_position(r, a, row, own, bad) * r.pairs + u.pair;
  if (u.axes == a * 0x01010101u) {
    const float4 x = reinterpret_cast<const float4*>(at)[0], y = reinterpret_cast<const float4*>(at)[1];
    w.t[0] = make_float2(x.x, x.y), w.t[1] = make_float2(x.z, x.w);
    w.t[2] = make_float2(y.x, y.y), w.t[3] = make_float2(y.z, y.w);
  } else {
    w.t[0] = at[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
      w.t[i] = r.table[(size_t)rope_position(r, (int)(u.axes >> 8 * i & 255), row, own, bad) * r.pairs + u.pair + i];
  }
  if (bad) atomicOr(r.status, kStatusBadIndex);
  return w;
}

// Every product, sum and difference rounded by itself. (Packed products and sums, two pairs an instruction, are made
// into fmas by the compiler, whatever their rounding is said to be.)
__device__ __forceinline__ void rope_pair(float& x, float& y, float2 t) {
  const float a = __fsub_rn(__fmul_rn(x, t.x), __fmul_rn(y, t.y));
  y = __fadd_rn(__fmul_rn(y, t.x), __fmul_rn(x, t.y));
  x = a;
}
__device__ __forceinline__ void rope_rotate(const RopeView& r, const RopeUnit& u, const RopeTurn& w, float (&x)[8]) {
  if (u.pair < 0) return;
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) rope_pair(x[2 * i], x[2 * i + 1], w.t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) rope_pair(x[i], x[4 + i], w.t[i]);
  }
}

// ---------------------------------------------------------------- the norm
// A number as the sum of two float32 ones, the second within half a step of the first
// (Dekker 1971, Knuth's two-sum): some 45 bits.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two two_add(const Two& a, const Two& b) {
  const Two s = two_sum(a.hi, b.hi);
  return Two{s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo))};
}
// The sum of a unit's squares, of `by` times its values; two at a time, each half with its own sum and what rounding took: exactly, also where
// the compiler makes a square and a sum one fma. (Squares of 16-bit numbers are exact.)
template <bool EXACT>
__device__ __forceinline__ Two squares_of(float (&x)[8], float by) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= by;
  float2 sum = __fmul2_rn(make_float2(x[0], x[1]), make_float2(x[0], x[1])), low = make_float2(0.f, 0.f);
  if (!EXACT) low = __ffma2_rn(make_float2(x[0], x[1]), make_float2(x[0], x[1]), make_float2(-sum.x, -sum.y));
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    const float2 y = make_float2(x[i], x[i + 1]), p = __fmul2_rn(y, y);
    const float2 s = __fadd2_rn(sum, p), t = __fadd2_rn(s, make_float2(-sum.x, -sum.y));
    const float2 u = __fadd2_rn(s, make_float2(-t.x, -t.y));
    low = __fadd2_rn(low, __fadd2_rn(__fadd2_rn(sum, make_float2(-u.x, -u.y)), __fadd2_rn(p, make_float2(-t.x, -t.y))));
    if (!EXACT) low = __fadd2_rn(low, __ffma2_rn(y, y, make_float2(-p.x, -p.y)));
    sum = s;
  }
  return two_add(Two{sum.x, low.x}, Two{sum.y, low.y});
}
// f32(1 / sqrt(mean)), mean = sum / n + eps, inv_n = f32(1 / n): the quotient's residual by fma; one step of Newton's from the
// approximation's 22 bits, its residual by fma. Where `mean` is within 2^+-100; elsewhere squares, sums or residuals leave float32.
__device__ __forceinline__ float rope_inverse_rms(const Two& sum, float n, float inv_n, float eps, float& mean) {
  const float q = __fmul_rn(sum.hi, inv_n);
  const Two m = two_add(two_sum(q, __fmul_rn(__fadd_rn(__fmaf_rn(-q, n, sum.hi), sum.lo), inv_n)), Two{eps, 0.f});
  const float s = __fadd_rn(m.hi, m.lo), low = __fadd_rn(__fsub_rn(m.hi, s), m.lo);
  const float y = rsqrtf(s), p = __fmul_rn(y, y), e = __fmaf_rn(y, y, -p);
  const float t = __fmaf_rn(-s, e, __fmaf_rn(-s, p, 1.f)) - low * p;
  mean = s;
  return __fmaf_rn(__fmul_rn(y, 0.5f), t, y);
}
// What a lane has of a head: EACH units, zeros where it has none.
template <typename T, int EACH>
struct HeadPart {
  Vec8<T> v[EACH];
};
// The sum of squares of `by` times a part's values.
template <typename T, int EACH>
__device__ __forceinline__ Two squares_of(const HeadPart<T, EACH>& x, float by) {
  Two sum;
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    float y[8];
    values8(x.v[e], y);
    const Two z = squares_of<sizeof(T) == 2>(y, by);
    sum = e ? two_add(sum, z) : z;
  }
  return sum;
}
__device__ __forceinline__ Two shfl_xor(const Two& x, int o) {
  return Two{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
}
// The inverse root of a head whose mean is out of rope_inverse_rms's range: of the head divided by a power of two, next
// to its largest magnitude or to eps's root. (Not inlined: its registers would be the callers' everywhere.)
template <int LANES, typename T, int EACH>
static __device__ __noinline__ float rope_inverse_rms_scaled(HeadPart<T, EACH> x, float n, float inv_n, float eps) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    float y[8];
    values8(x.v[e], y);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[i]));
  }
#pragma unroll
  for (int o = 1; o < LANES; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int of_top = (int)(__float_as_uint(top) >> 23) - 127;
  const int of_eps = eps > 0.f ? ((int)(__float_as_uint(eps) >> 23) - 126) >> 1 : -126;
  const float down = __uint_as_float((uint32_t)(127 - min(max(max(of_top, of_eps), -126), 126)) << 23);
  Two sum = squares_of(x, down);
#pragma unroll
  for (int o = 1; o < LANES; o *= 2) sum = two_add(sum, shfl_xor(sum, o));
  float mean;
  return rope_inverse_rms(sum, n, inv_n, eps * down * down, mean) * down;
}
__device__ __forceinline__ bool rope_out_of_range(float mean) { return !(mean >= 0x1p-100f && mean <= 0x1p100f); }
// The inverse root of one head, of any magnitude, each lane of a group of LANES with a part of it.
template <int LANES, typename T, int EACH>
__device__ __forceinline__ float rope_inverse_rms_of(const HeadPart<T, EACH>& x, float n, float inv_n, float eps) {
  Two sum = squares_of(x, 1.f);
#pragma unroll
  for (int o = 1; o < LANES; o *= 2) sum = two_add(sum, shfl_xor(sum, o));
  float mean;
  const float r = rope_inverse_rms(sum, n, inv_n, eps, mean), scaled = rope_inverse_rms_scaled<LANES>(x, n, inv_n, eps);
  return rope_out_of_range(mean) ? scaled : r;
}
// rope_inverse_rms of four heads, each lane of a group of LANES with a part of each one: two
// steps hand half of the heads to the neighbour, so that each lane goes on with one head and takes one root
// (5 sums of two numbers instead of 16 for 16 lanes). All lanes of the warp call it. Whether the lane's own head is out of range.
template <int LANES, typename T, int EACH>
__device__ __forceinline__ bool rope_inverse_rms4(const HeadPart<T, EACH> (&x)[4], float n, float inv_n, float eps,
                                                  float (&inv)[4]) {
  const int lane = threadIdx.x & 31;
  const bool b0 = lane & 1, b1 = lane & 2;
  Two s[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) s[h] = squares_of(x[h], 1.f);
  const Two u = two_add(b0 ? s[2] : s[0], shfl_xor(b0 ? s[0] : s[2], 1)), w = two_add(b0 ? s[3] : s[1], shfl_xor(b0 ? s[1] : s[3], 1));
  Two z = two_add(b1 ? w : u, shfl_xor(b1 ? u : w, 2));
#pragma unroll
  for (int o = 4; o < LANES; o *= 2) z = two_add(z, shfl_xor(z, o));
  float mean;
  const float r = rope_inverse_rms(z, n, inv_n, eps, mean);
  const bool far = rope_out_of_range(mean);
#pragma unroll
  for (int h = 0; h < 4; ++h) inv[h] = __shfl_sync(0xffffffffu, r, (lane & ~3) | h >> 1 | (h & 1) << 1);
  return far;
}
// The same, and those heads that are out of its range again.
template <int LANES, typename T, int EACH>
__device__ __forceinline__ void rope_inverse_rms4_of_any(const HeadPart<T, EACH> (&x)[4], float n, float inv_n, float eps, float (&inv)[4]) {
  const bool far = rope_inverse_rms4<LANES>(x, n, inv_n, eps, inv);
  if (!__any_sync(0xffffffffu, far)) return;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const bool mine = __shfl_sync(0xffffffffu, far, (threadIdx.x & 28) | h >> 1 | (h & 1) << 1);
    const float again = rope_inverse_rms_scaled<LANES>(x[h], n, inv_n, eps);
    if (mine) inv[h] = again;
  }
}

// ---------------------------------------------------------------- elements
__device__ __forceinline__ Vec8<float> load44(const float* p, int d0, int d1) {
  return Vec8<float>{*reinterpret_cast<const float4*>(p + d0), *reinterpret_cast<const float4*>(p + d1)};
}
template <typename T>
__device__ __forceinline__ Vec8<T> load44(const T* p, int d0, int d1) {
  const uint2 a = *reinterpret_cast<const uint2*>(p + d0), b = *reinterpret_cast<const uint2*>(p + d1);
  return Vec8<T>{make_uint4(a.x, a.y, b.x, b.y)};
}
__device__ __forceinline__ void store44(float* p, int d0, int d1, const Vec8<float>& e) {
  *reinterpret_cast<float4*>(p + d0) = e.a;
  *reinterpret_cast<float4*>(p + d1) = e.b;
}
template <typename T>
__device__ __forceinline__ void store44(T* p, int d0, int d1, const Vec8<T>& e) {
  *reinterpret_cast<uint2*>(p + d0) = make_uint2(e.a.x, e.a.y);
  *reinterpret_cast<uint2*>(p + d1) = make_uint2(e.a.z, e.a.w);
}
template <typename T>
__device__ __forceinline__ Vec8<T> vec8_of(const float (&x)[8]) {
  if constexpr (sizeof(T) == 4)
    return Vec8<T>{make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7])};
  else
    return Vec8<T>{make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]))};
}

// What stands for a head that is not there: one whose norm takes no second look.
template <typename T>
__device__ __forceinline__ Vec8<T> ones8() {
  const float x[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  return vec8_of<T>(x);
}

// Norm and rotation of a unit's values, w its norm weights.
__device__ __forceinline__ void rope_norm(float (&x)[8], float inv, const float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 y = __fmul2_rn(__fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(inv, inv)), make_float2(w[i], w[i + 1]));
    x[i] = y.x, x[i + 1] = y.y;
  }
}

// ---------------------------------------------------------------- rows into rows
// Heads that a group of lanes does of one row: all, or as few as it takes to have `want` groups.
inline int rope_heads_a_group(long long rows, int heads, long long want) {
  int each = heads;
  while (each > 1 && rows * ((heads + each - 1) / each) < want) each = (each + 1) / 2;
  return each;
}

// The row of group `group`, which may be past the last one.
__device__ __forceinline__ long long rope_row_of(const RopeRows& a, long long group) {
  return group / ((a.heads + a.heads_a_group - 1) / a.heads_a_group);
}
// The heads of rope_rows_group from its i-th on, one after the other and of any magnitude. (Not inlined: its registers
// would be rope_rows_group's: 16390 rows of 32 heads of 128 64 us instead of 61, 59.9 without any of this.)
template <typename T, int LANES, int EACH>
static __device__ __noinline__ void rope_rows_rest(const RopeView& r, const RopeRows& a, int row, int own, int lane, int h0, int h1, int i) {
  RopeUnit unit[EACH];
  RopeTurn turn[EACH];
  float w[EACH][8];
  bool mine[EACH];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    mine[e] = (lane + e * LANES) * 8 < a.dim && h0 < h1;
    unit[e] = rope_unit(r, mine[e] ? lane + e * LANES : 0);
    if (mine[e]) turn[e] = rope_turn(r, unit[e], row, own);
    const Vec8<float> v = load44(a.norm, unit[e].d0, unit[e].d1);
    values8(v, w[e]);
  }
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  T* out = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll 1
  for (; i < a.heads_a_group; ++i) {
    const bool here = h0 + i < h1;
    HeadPart<T, EACH> part = {};
#pragma unroll
    for (int e = 0; e < EACH; ++e)
      if (mine[e] && here) part.v[e] = load44(x + (size_t)(h0 + i) * a.dim, unit[e].d0, unit[e].d1);
    const float inv = rope_inverse_rms_of<LANES>(part, (float)a.dim, 1.f / (float)a.dim, a.eps);
#pragma unroll
    for (int e = 0; e < EACH; ++e)
      if (mine[e] && here) {
        float y[8];
        values8(part.v[e], y);
        rope_norm(y, inv, w[e]);
        rope_rotate(r, unit[e], turn[e], y);
        store44(out + (size_t)(h0 + i) * a.dim, unit[e].d0, unit[e].d1, vec8_of<T>(y));
      }
  }
}
// Group `group` of LANES lanes does heads_a_group heads of one row, EACH units a
// lane; `lane` within the group; nothing of a row that is not `live`. All lanes of the warp call it.
template <typename T, int LANES, int EACH>
__device__ __forceinline__ void rope_rows_group(const RopeView& r, const RopeRows& a, long long group, int lane,
                                                int own, bool live) {
  constexpr int BATCH = 4;  // heads whose values are on their way together
  const int per_row = (a.heads + a.heads_a_group - 1) / a.heads_a_group;
  live = live && group / per_row < a.num_rows;
  const long long row = live ? group / per_row : 0;
  const int h0 = (int)(group % per_row) * a.heads_a_group, h1 = live ? min(h0 + a.heads_a_group, a.heads) : h0;
  const float inv_dim = 1.f / (float)a.dim;
  RopeUnit unit[EACH];
  RopeTurn turn[EACH];
  float w[EACH][8];
  bool mine[EACH];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    mine[e] = (lane + e * LANES) * 8 < a.dim && h0 < h1;
    unit[e] = rope_unit(r, mine[e] ? lane + e * LANES : 0);
    if (mine[e]) turn[e] = rope_turn(r, unit[e], (int)row, own);
    if (mine[e] && a.norm) {
      const Vec8<float> v = load44(a.norm, unit[e].d0, unit[e].d1);
      values8(v, w[e]);
    }
  }
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  T* out = static_cast<T*>(a.out) + row * a.ldo;
  for (int i = 0; i < a.heads_a_group; i += BATCH) {
    Vec8<T> v[BATCH][EACH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
#pragma unroll
      for (int e = 0; e < EACH; ++e)
        if (mine[e] && h0 + i + j < h1) v[j][e] = load44(x + (size_t)(h0 + i + j) * a.dim, unit[e].d0, unit[e].d1);
    float inv[BATCH];
    if (a.norm) {
      HeadPart<T, EACH> part[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
#pragma unroll
        for (int e = 0; e < EACH; ++e) part[j].v[e] = h0 + i + j >= h1 ? ones8<T>() : (mine[e] ? v[j][e] : Vec8<T>{});
      if (__any_sync(0xffffffffu, rope_inverse_rms4<LANES>(part, (float)a.dim, inv_dim, a.eps, inv)))
        return rope_rows_rest<T, LANES, EACH>(r, a, (int)row, own, lane, h0, h1, i);
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
#pragma unroll
      for (int e = 0; e < EACH; ++e)
        if (mine[e] && h0 + i + j < h1) {
          float y[8];
          values8(v[j][e], y);
          if (a.norm) rope_norm(y, inv[j], w[e]);
          rope_rotate(r, unit[e], turn[e], y);
          store44(out + (size_t)(h0 + i + j) * a.dim, unit[e].d0, unit[e].d1, vec8_of<T>(y));
        }
  }
}

}  // namespace apr
