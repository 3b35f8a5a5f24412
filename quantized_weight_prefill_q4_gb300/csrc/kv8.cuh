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

// Every kernel of the cache is launched before the work ahead of it is done
// and waits here for it. What it reads before are the index arrays alone (lens,
// row_start, page_table): no kernel of the library writes those but the
// eviction's, which let nothing start before they have ended, and a kernel
// that lets the next one start early does so after its own wait, so that all
// work but its own is done by then.
__device__ __forceinline__ void kv8_ready() { grid_dependency_wait(); }

__device__ __forceinline__ void kv8_flag(const Kv8View& v) { atomicOr(v.status, kStatusBadIndex); }

// Tokens of sequence b, within 0 .. max_len whatever the array says.
__device__ __forceinline__ int kv8_len(const Kv8View& v, int b) {
  const int n = v.lens[b];
  if (n >= 0 && n <= v.max_len) return n;
  kv8_flag(v);
  return n < 0 ? 0 : v.max_len;
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
template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// N consecutive elements on a 16-byte boundary (N * sizeof(T) a multiple of 16)
template <typename T, int N>
struct alignas(16) Elems {
  T x[N];
};

// ---------------------------------------------------------------- codes
// The scale of a page and head whose largest finite magnitude is amax: the
// same float32 value whether the quotient is taken in 32 or in 64 bits.
__device__ __forceinline__ float kv8_scale_of(float amax) { return __fdiv_rn(amax, 127.0f); }

// |x| where it is finite, else 0.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.f;
}

// x / s decided in 64 bits. A quotient of two float32 values that is not a
// half itself is further from one than 64-bit division rounds by.
static __device__ __noinline__ float kv8_round_exact(float x, float s) {
  return (float)fmin(fmax(rint((double)x / (double)s), -127.0), 127.0);
}

// rint(x / s) clamped to +-127, inv = 1 / s. The float32 product x * inv is
// within 3e-5 of the quotient; only where that leaves the rounding open (one
// value in about 5000) is the quotient taken in 64 bits.
__device__ __forceinline__ int kv8_code(float x, float s, float inv) {
  if (!(s > 0.f)) return 0;
  const float f = x * inv;
  if (!(fabsf(f) < 128.f) || s < 1e-37f)  // infinities, NaN, scales whose reciprocal is not a normal number
    return x != x ? 0 : (fabsf(x) <= FLT_MAX ? (int)kv8_round_exact(x, s) : (x > 0.f ? 127 : -127));
  float r = rintf(f);
  if (fabsf(f - r) > 0.4999f) r = kv8_round_exact(x, s);
  return (int)fminf(fmaxf(r, -127.f), 127.f);
}

// Four codes as one word, the first in the lowest byte.
__device__ __forceinline__ uint32_t kv8_pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 255) | ((uint32_t)(b & 255) << 8) | ((uint32_t)(c & 255) << 16) | ((uint32_t)d << 24);
}
// Byte i of a word of codes, as a signed number.
__device__ __forceinline__ int kv8_byte(uint32_t w, int i) { return (int)(int8_t)(w >> (8 * i)); }

}  // namespace apr
