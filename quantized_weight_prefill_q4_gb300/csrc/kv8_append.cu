// Rows into and out of the 8-bit paged KV cache (include/apr_kv8.h).
//
// Append. One CTA per (page that gets rows, KV head, K or V): it finds the
// largest magnitude of the page's new rows, raises the page's scale if that
// asks for more, re-rounds what the page held if it was raised, and writes the
// new codes. The block of a scale is one CTA's whole work, so no two CTAs
// share a scale and the result does not depend on their order. Bound by
// memory: a row is read once (its first 32 values a thread stay in registers
// between the two passes, longer pages come from L1 the second time) and one
// byte a value written.
//
// Read. One CTA per (run of at most 128 tokens within a page, KV head, K or
// V); a thread's 16-byte stores cover neighbouring elements of a row.

#include "apr_internal.h"
#include "host_common.h"
#include "kv8.cuh"

namespace apr {
namespace {

constexpr int A_THREADS = 256;
constexpr int A_HELD = 4;  // vectors of 8 values a thread keeps between the passes

template <typename T>
__device__ __forceinline__ float amax_of(const Elems<T, 8>& e, float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(to_f32<T>(e.x[i])));
  return m;
}

template <typename T>
__device__ __forceinline__ uint2 codes_of(const Elems<T, 8>& e, float s, float inv) {
  int c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = kv8_code(to_f32<T>(e.x[i]), s, inv);
  return make_uint2(kv8_pack4(c[0], c[1], c[2], c[3]), kv8_pack4(c[4], c[5], c[6], c[7]));
}

template <typename T>
__global__ void __launch_bounds__(A_THREADS) kv8_append_kernel(Kv8View v, const T* __restrict__ k,
                                                               const T* __restrict__ vv, long long ld) {
  __shared__ float s_max[A_THREADS / 32];
  const int b = blockIdx.z, g = (int)(blockIdx.x % v.kv_heads), slot = (int)(blockIdx.x / v.kv_heads);
  const bool is_v = blockIdx.y != 0;
  const int len = kv8_len(v, b);
  const Kv8Span span = kv8_rows(v, b);
  const int first = len - span.n;  // position of row r0; rows of negative positions are skipped
  if (span.n == 0 || len == 0) return;
  const int index = (max(first, 0) >> v.page_shift) + slot;
  if (index > (len - 1) >> v.page_shift) return;
  const int page = kv8_page(v, b, index);
  if (page < 0) return;
  kv8_ready();
  grid_launch_dependents();
  const int page0 = index << v.page_shift;
  const int lo = max(max(first, 0), page0), hi = min(len, page0 + (1 << v.page_shift));
  const int held = lo - page0;
  const int vshift = 31 - __clz(v.dim / 8);  // vectors of 8 values a row
  const T* src = (is_v ? vv : k) + (long long)(span.r0 + lo - first) * ld + (size_t)g * v.dim;
  int8_t* codes = (is_v ? v.V : v.K) + kv8_codes_at(v, page, g);
  float* scale = (is_v ? v.v_scale : v.k_scale) + kv8_scale_at(v, page, g);
  const float s_old = held > 0 ? *scale : 0.f;
  const int nvec = (hi - lo) << vshift;
  const int cmask = (1 << vshift) - 1;
  auto at = [&](int i) {
    return reinterpret_cast<const Elems<T, 8>*>(src + (long long)(i >> vshift) * ld + (i & cmask) * 8);
  };

  // ---- the largest magnitude
  Elems<T, 8> keep[A_HELD];
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < A_HELD; ++j) {
    const int i = threadIdx.x + j * A_THREADS;
    if (i < nvec) keep[j] = *at(i);
  }
#pragma unroll
  for (int j = 0; j < A_HELD; ++j)
    if ((int)threadIdx.x + j * A_THREADS < nvec) m = amax_of<T>(keep[j], m);
#pragma unroll 4
  for (int i = threadIdx.x + A_HELD * A_THREADS; i < nvec; i += A_THREADS) m = amax_of<T>(*at(i), m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < A_THREADS / 32; ++w) m = fmaxf(m, s_max[w]);

  // ---- the scale, and what the page held under a raised one
  const float s = fmaxf(s_old, kv8_scale_of(m));
  const float inv = __fdiv_rn(1.0f, s);
  if (threadIdx.x == 0 && (held == 0 || s > s_old)) *scale = s;
  if (held > 0 && s > s_old) {
    uint4* old = reinterpret_cast<uint4*>(codes);
    for (int i = threadIdx.x; i < held * v.dim / 16; i += A_THREADS) {
      uint4 w = old[i];
      uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        int c[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) c[t] = kv8_code((float)kv8_byte(u[j], t) * s_old, s, inv);
        u[j] = kv8_pack4(c[0], c[1], c[2], c[3]);
      }
      old[i] = w;
    }
  }

  // ---- the new codes
  uint2* dst = reinterpret_cast<uint2*>(codes + (size_t)held * v.dim);
#pragma unroll
  for (int j = 0; j < A_HELD; ++j) {
    const int i = threadIdx.x + j * A_THREADS;
    if (i < nvec) dst[i] = codes_of<T>(keep[j], s, inv);
  }
  for (int i = threadIdx.x + A_HELD * A_THREADS; i < nvec; i += A_THREADS) dst[i] = codes_of<T>(*at(i), s, inv);
}

// ---------------------------------------------------------------- read
constexpr int R_THREADS = 256;

// tokens of a CTA's run: a page's, at most 128
__host__ __device__ inline int read_run_shift(int page_shift) { return page_shift < 7 ? page_shift : 7; }

template <typename T>
__global__ void __launch_bounds__(R_THREADS) kv8_read_kernel(Kv8View v, T* __restrict__ k, T* __restrict__ vv,
                                                             long long ld) {
  constexpr int N = 16 / sizeof(T);  // values of a 16-byte store
  const int b = blockIdx.z, g = (int)(blockIdx.x % v.kv_heads), run = (int)(blockIdx.x / v.kv_heads);
  const bool is_v = blockIdx.y != 0;
  const int len = kv8_len(v, b);
  const Kv8Span span = kv8_rows(v, b);
  if (span.n == 0) return;
  const int first = len - span.n;
  const int rshift = read_run_shift(v.page_shift);
  const int vshift = 31 - __clz(v.dim / N), cmask = (1 << vshift) - 1;
  T* out = (is_v ? vv : k) + (long long)span.r0 * ld + (size_t)g * v.dim;
  const int index = (max(first, 0) >> rshift) + run;
  kv8_ready();
  grid_launch_dependents();
  if (run == 0 && first < 0) {  // rows before the sequence's start
    Elems<T, N> zero;
#pragma unroll
    for (int t = 0; t < N; ++t) zero.x[t] = from_f32<T>(0.f);
    for (int i = threadIdx.x; i < (min(-first, span.n) << vshift); i += R_THREADS)
      *reinterpret_cast<Elems<T, N>*>(out + (long long)(i >> vshift) * ld + (i & cmask) * N) = zero;
  }
  const int lo = max(max(first, 0), index << rshift), hi = min(len, (index + 1) << rshift);
  if (lo >= hi) return;
  const int page = kv8_page(v, b, lo >> v.page_shift);
  if (page < 0) return;
  const float s = (is_v ? v.v_scale : v.k_scale)[kv8_scale_at(v, page, g)];
  const int8_t* codes = (is_v ? v.V : v.K) + kv8_codes_at(v, page, g) +
                        (size_t)(lo & ((1 << v.page_shift) - 1)) * v.dim;
  out += (long long)(lo - first) * ld;
#pragma unroll 4
  for (int i = threadIdx.x; i < (hi - lo) << vshift; i += R_THREADS) {
    uint32_t w[N / 4];
    if (N == 4)
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
    else
      *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(codes) + i);
    Elems<T, N> e;
#pragma unroll
    for (int t = 0; t < N; ++t) e.x[t] = from_f32<T>((float)kv8_byte(w[t / 4], t % 4) * s);
    *reinterpret_cast<Elems<T, N>*>(out + (long long)(i >> vshift) * ld + (i & cmask) * N) = e;
  }
}

template <typename T>
cudaError_t append_typed(const Kv8View& v, const void* k, const void* vv, long long ld, cudaStream_t s) {
  // pages that max_rows rows can touch
  const int page = 1 << v.page_shift, slots = (int)(((long long)v.max_rows + page - 2) / page + 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)slots * v.kv_heads, 2, (unsigned)v.num_seqs);
  cfg.blockDim = dim3(A_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_append_kernel<T>, v, (const T*)k, (const T*)vv, ld);
}

template <typename T>
cudaError_t read_typed(const Kv8View& v, void* k, void* vv, long long ld, cudaStream_t s) {
  const int run = 1 << read_run_shift(v.page_shift), runs = (int)(((long long)v.max_rows + run - 2) / run + 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)runs * v.kv_heads, 2, (unsigned)v.num_seqs);
  cfg.blockDim = dim3(R_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_read_kernel<T>, v, (T*)k, (T*)vv, ld);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8View& v, int type, const void* k, const void* vv, long long ld,
                              cudaStream_t s) {
  if (type == APR_T_F32) return append_typed<float>(v, k, vv, ld, s);
  if (type == APR_T_F16) return append_typed<__half>(v, k, vv, ld, s);
  return append_typed<__nv_bfloat16>(v, k, vv, ld, s);
}

cudaError_t launch_kv8_read(const Kv8View& v, int type, void* k, void* vv, long long ld, cudaStream_t s) {
  if (type == APR_T_F32) return read_typed<float>(v, k, vv, ld, s);
  if (type == APR_T_F16) return read_typed<__half>(v, k, vv, ld, s);
  return read_typed<__nv_bfloat16>(v, k, vv, ld, s);
}

}  // namespace apr
