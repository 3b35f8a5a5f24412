// What the append to the 8-bit paged KV cache (kv8_append.cu) shares with the one
// that rotates k on the way (rope_append.cu).
#pragma once

#include "host_common.h"
#include "kv8.cuh"

namespace apr {

constexpr int A_THREADS = 128;
constexpr int A_WARPS = A_THREADS / 32;

// The largest magnitude; NaN is passed over, an infinity is not (the caller
// looks again then, finite values only).
__device__ __forceinline__ float amax_of(const Vec8<float>& e, float m) {
  m = fmaxf(m, fmaxf(fmaxf(fabsf(e.a.x), fabsf(e.a.y)), fmaxf(fabsf(e.a.z), fabsf(e.a.w))));
  return fmaxf(m, fmaxf(fmaxf(fabsf(e.b.x), fabsf(e.b.y)), fmaxf(fabsf(e.b.z), fabsf(e.b.w))));
}
template <typename T2>
__device__ __forceinline__ float amax_of_pairs(const uint4& w, float m) {
  const T2* h = reinterpret_cast<const T2*>(&w);
  const T2 t = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
  return fmaxf(m, fmaxf(__low2float(t), __high2float(t)));
}
__device__ __forceinline__ float amax_of(const Vec8<__half>& e, float m) { return amax_of_pairs<__half2>(e.a, m); }
__device__ __forceinline__ float amax_of(const Vec8<__nv_bfloat16>& e, float m) {
  return amax_of_pairs<__nv_bfloat162>(e.a, m);
}
template <typename T>
__device__ __forceinline__ float finite_amax_of(const Vec8<T>& e, float m) {
  float x[8];
  values8(e, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(x[i]));
  return m;
}

template <typename T>
__device__ __forceinline__ uint2 codes_of(const Vec8<T>& e, const Kv8Scale& s) {
  float x[8];
  values8(e, x);
  return kv8_codes8(x, s);
}

// The largest value over the CTA.
template <int WARPS>
__device__ __forceinline__ float block_max(float m, float* warp_max) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) m = fmaxf(m, warp_max[w]);
  return m;
}

// The first of a sequence's units, one for each page that its rows may go to: n
// rows touch at most n / page_tokens + 2 pages, so this many further on begins the next
// one's, and a CTA finds its sequence by a search instead of adding up all of them
// (2 rows of each of 16384 sequences: 0.6 ms, 10.8 when every CTA did).
__device__ __forceinline__ int first_append_unit(const Kv8View& v, int b) {
  return (v.row_start[b] >> v.page_shift) + 2 * b;
}

// Heads of a CTA: all, or as few as it takes to give every SM `most` CTAs.
inline int heads_a_cta(long long units, int kv_heads, int most) {
  const long long want = (long long)most * num_sms() / (2 * units > 0 ? 2 * units : 1);  // CTAs of a unit, K or V
  return want <= 1 ? kv_heads : (int)(want >= kv_heads ? 1 : (kv_heads + want - 1) / want);
}

}  // namespace apr
