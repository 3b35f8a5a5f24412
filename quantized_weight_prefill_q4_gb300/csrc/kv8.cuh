// The 8-bit paged KV cache (include/apr_kv8.h) as its kernels see it: where a
// token's codes lie, which rows a call is about, the checks of what the device
// arrays say, and the quantisation to codes.
#pragma once

#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "apr_kv8.h"
#include "dev_common.cuh"

namespace apr {

struct Kv8View {
  int8_t* K;
  int8_t* V;
  float* k_scale;
  float* v_scale;
  const int* table;
  const int* lens;
  const int* row_start;  // nullptr: one row a sequence
  unsigned* status;
  int num_pages, kv_heads, page_shift, dim;
  int table_ld, num_seqs, num_rows, max_rows, max_len;
};

__device__ __forceinline__ void kv8_flag(const Kv8View& v) { atomicOr(v.status, kStatusBadIndex); }

// Tokens of sequence b, within 0 .. max_len. Any other length counts as 0, not
// as the nearest one: rows appended behind max_len tokens of a sequence that
// claims more would overwrite tokens that it holds.
__device__ __forceinline__ int kv8_len(const Kv8View& v, int b) {
  const int n = v.lens[b];
  if ((unsigned)n <= (unsigned)v.max_len) return n;
  kv8_flag(v);
  return 0;
}

// The call's rows of sequence b: n of them from packed row r0 on, within the
// call's rows whatever the array says.
struct Kv8Span {
  int r0, n;
};
__device__ __forceinline__ Kv8Span kv8_rows(const Kv8View& v, int b) {
  if (!v.row_start) return Kv8Span{b, 1};
  const int a = v.row_start[b], e = v.row_start[b + 1];
  if (a >= 0 && e >= a && e <= v.num_rows && e - a <= v.max_rows) return Kv8Span{a, e - a};
  kv8_flag(v);
  return Kv8Span{0, 0};
}

// The last of the sequences that `begins` says yes of, where it does of all before
// one and of none from there on; 0 if of none. (Within 0 .. num_seqs - 1 whatever it
// says.) Found by the whole warp, 128 candidates at a time,
// whose loads are under way together (an append to 64 sequences 5.3 us, 5.5 with 32).
template <typename F>
__device__ __forceinline__ int kv8_last_sequence(const Kv8View& v, const F& begins) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  for (int n = v.num_seqs; n > 1;) {  // one of lo .. lo + n - 1
    const int step = (n + 127) / 128;
    int count = 0;
#pragma unroll
    for (int i = 0; i < 128; i += 32) {
      const bool yes = (i + lane) * step < n && begins(lo + (i + lane) * step);
      count += __popc(__ballot_sync(0xffffffffu, yes));
    }
    const int last = max(count - 1, 0) * step;
    lo += last;
    n = min(step, n - last);
  }
  return lo;
}
// The sequence that packed row `row` belongs to, if any.
__device__ __forceinline__ int kv8_sequence_of(const Kv8View& v, int row) {
  return v.row_start ? kv8_last_sequence(v, [&](int b) { return v.row_start[b] <= row; }) : row;
}

// The page of sequence b's tokens `index << page_shift` on, or -1 (flagged)
// where the table names none.
__device__ __forceinline__ int kv8_page(const Kv8View& v, int b, int index) {
  const int p = v.table[(size_t)b * v.table_ld + index];
  if (p >= 0 && p < v.num_pages) return p;
  kv8_flag(v);
  return -1;
}

// Offset of the codes of (page, head), and of its scale.
__device__ __forceinline__ size_t kv8_scale_at(const Kv8View& v, int page, int g) {
  return (size_t)page * v.kv_heads + g;
}
__device__ __forceinline__ size_t kv8_codes_at(const Kv8View& v, int page, int g) {
  return (kv8_scale_at(v, page, g) << v.page_shift) * v.dim;
}

// ---------------------------------------------------------------- elements
// Eight consecutive elements of a row, on a 16-byte boundary.
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
  float4 a, b;
};
template <>
struct Vec8<__half> {
  uint4 a;
};
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
};
__device__ __forceinline__ Vec8<float> load8(const float* p) {
  const float4* q = reinterpret_cast<const float4*>(p);
  return Vec8<float>{q[0], q[1]};
}
__device__ __forceinline__ Vec8<__half> load8(const __half* p) {
  return Vec8<__half>{*reinterpret_cast<const uint4*>(p)};
}
__device__ __forceinline__ Vec8<__nv_bfloat16> load8(const __nv_bfloat16* p) {
  return Vec8<__nv_bfloat16>{*reinterpret_cast<const uint4*>(p)};
}
__device__ __forceinline__ void values8(const Vec8<float>& e, float (&x)[8]) {
  x[0] = e.a.x, x[1] = e.a.y, x[2] = e.a.z, x[3] = e.a.w;
  x[4] = e.b.x, x[5] = e.b.y, x[6] = e.b.z, x[7] = e.b.w;
}
__device__ __forceinline__ void values8(const Vec8<__half>& e, float (&x)[8]) {
  const uint32_t w[4] = {e.a.x, e.a.y, e.a.z, e.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void values8(const Vec8<__nv_bfloat16>& e, float (&x)[8]) {
  const uint32_t w[4] = {e.a.x, e.a.y, e.a.z, e.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

// Two float32 values as two 16-bit ones.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------- fp16
// Two codes, plus 128, from the bytes that `sel` picks: 0x64uu is the fp16
// number 1024 + uu.
__device__ __forceinline__ uint32_t half2_of_codes(uint32_t biased, uint32_t sel) {
  const uint32_t h = __byte_perm(biased, 0x64646464u, sel);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&x);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half2_values(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- codes
// The scale of a page and head whose largest finite magnitude is amax: the
// same float32 value whether the quotient is taken in 32 or in 64 bits.
__device__ __forceinline__ float kv8_scale_of(float amax) { return __fdiv_rn(amax, 127.0f); }

// |x| where it is finite, else 0.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.f;
}

// rint(x / s) clamped to +-127; NaN 0, infinities +-127, 0 under s = 0. The
// quotient is taken in 64 bits: one of two float32 values that is not a half
// itself is further from one than 64-bit division rounds by.
static __device__ __noinline__ uint32_t kv8_code(float x, float s) {
  if (!(s > 0.f) || x != x) return 0;
  return (uint32_t)(int)fmin(fmax(rint((double)x / (double)s), -127.0), 127.0);
}

// Bytes i and i + 1 of a word, exclusive-or'ed with 0x80808080, as float32
// values: 2^23 + (code + 128) less what was added.
__device__ __forceinline__ float2 kv8_bytes_f32(uint32_t biased, int i) {
  return __fadd2_rn(make_float2(__uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7540u + i)),
                                __uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7541u + i))),
                    make_float2(-8388736.f, -8388736.f));
}

// A scale with what rounding under it takes. (Halves and reciprocals of the
// smallest numbers are not exact, or not numbers: half = -1 leaves all to kv8_code.)
struct Kv8Scale {
  float s, inv, half;
};
__device__ __forceinline__ Kv8Scale kv8_rounding_to(float s) {
  return Kv8Scale{s, __fdiv_rn(1.0f, s), s >= 1e-37f ? 0.5f * s : -1.f};
}

// The fast way to rint(x / s), two values at a time: x * (1 / s) added to
// 1.5 * 2^23 rounds to a whole number w, and the sum's low byte is the code.
// Where w is nearest to the exact quotient, x - w s is less than s / 2, and one
// fma gives it exactly (it is a multiple of half the scale's last bit, below
// 2^24 of them). `open` says where it is not less, or not a number: a tie, or a
// product that rounded across one (one float32 value in 10^5, but one bf16 value
// in 200, whose quotients by the largest of them often lie next to a half).
__device__ __forceinline__ uint2 kv8_round_sums(float2 x, const Kv8Scale& k, bool& open) {
  const float2 sum = __ffma2_rn(x, make_float2(k.inv, k.inv), make_float2(12582912.f, 12582912.f));
  const float2 w = __fadd2_rn(sum, make_float2(-12582912.f, -12582912.f));
  const float2 r = __ffma2_rn(w, make_float2(-k.s, -k.s), x);
  open |= !(fabsf(r.x) < k.half) || !(fabsf(r.y) < k.half);
  return make_uint2(__float_as_uint(sum.x), __float_as_uint(sum.y));
}
// The same settled: one more or less where x - w s is over s / 2, or at it and w odd.
__device__ __forceinline__ uint32_t kv8_round_settled(uint32_t sum, float x, const Kv8Scale& k) {
  if (!(k.half > 0.f && fabsf(x) <= FLT_MAX)) return kv8_code(x, k.s);
  const float r = fmaf(-(__uint_as_float(sum) - 12582912.f), k.s, x), a = fabsf(r);
  return a > k.half || (a == k.half && (sum & 1)) ? (r > 0.f ? sum + 1 : sum - 1) : sum;
}
// The low bytes of four words as one.
__device__ __forceinline__ uint32_t kv8_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Codes of eight values of magnitude up to 127 s (1 + 2^-23).
__device__ __forceinline__ uint2 kv8_codes8(const float (&x)[8], const Kv8Scale& k) {
  bool open = false;
  uint2 r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = kv8_round_sums(make_float2(x[2 * i], x[2 * i + 1]), k, open);
  if (open) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = make_uint2(kv8_round_settled(r[i].x, x[2 * i], k), kv8_round_settled(r[i].y, x[2 * i + 1], k));
  }
  return make_uint2(kv8_low_bytes(r[0].x, r[0].y, r[1].x, r[1].y), kv8_low_bytes(r[2].x, r[2].y, r[3].x, r[3].y));
}

// Four codes under the scale `from` as codes under k.s, of values of magnitude
// up to 127 s (1 + 2^-23): rint(float32(code * from) / s).
static __device__ __noinline__ uint32_t kv8_requantise4_settled(uint32_t biased, float from, Kv8Scale k) {
  bool open = false;
  uint2 r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = __fmul2_rn(kv8_bytes_f32(biased, 2 * i), make_float2(from, from));
    r[i] = kv8_round_sums(x, k, open);
    r[i] = make_uint2(kv8_round_settled(r[i].x, x.x, k), kv8_round_settled(r[i].y, x.y, k));
  }
  return kv8_low_bytes(r[0].x, r[0].y, r[1].x, r[1].y);
}
__device__ __forceinline__ uint32_t kv8_requantise4(uint32_t w, float from, const Kv8Scale& k) {
  const uint32_t biased = w ^ 0x80808080u;
  const float2 f = make_float2(from, from);
  bool open = false;
  const uint2 a = kv8_round_sums(__fmul2_rn(kv8_bytes_f32(biased, 0), f), k, open);
  const uint2 b = kv8_round_sums(__fmul2_rn(kv8_bytes_f32(biased, 2), f), k, open);
  return open ? kv8_requantise4_settled(biased, from, k) : kv8_low_bytes(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint4 kv8_requantise16(const uint4& w, float from, const Kv8Scale& k) {
  return make_uint4(kv8_requantise4(w.x, from, k), kv8_requantise4(w.y, from, k), kv8_requantise4(w.z, from, k),
                    kv8_requantise4(w.w, from, k));
}

}  // namespace apr
