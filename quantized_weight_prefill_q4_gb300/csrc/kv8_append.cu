// Rows into and out of the 8-bit paged KV cache (include/apr_kv8.h).
//
// Append. The block of a scale, a page of one head, is one CTA's work at a
// time, so no two CTAs share a scale and the result does not depend on their
// order: it finds the largest magnitude of the page's new rows, raises the
// page's scale if that asks for more, re-rounds what the page held if it was
// raised, and writes the new codes. A CTA takes several heads of the page one
// after the other, K or V: the way from the lengths over the table to the page
// is gone once, and the next head's rows are under way while one is rounded.
// The pages that a call may touch are numbered through, so that prompts of
// different lengths leave at most two CTAs a sequence (of each head) without work.
// Bound by memory: a row is read once (up to 32 registers a thread hold it
// between the two passes; what a larger page has more comes from L1 the second
// time) and one byte a value written; the rounding is five instructions and a
// byte permute a value (kv8_codes8).
//
// Measured (GB300): 13000 rows of 8 heads of 128 in bf16, 9 prompts: 22.8 us, 80 MB
// (0.52 of the HBM rate); 50001 of 8 heads of 64 in fp16: 34.1 us, 154 MB (0.67); the 13000
// rows of 4 heads of 256 in float32: 32.4 us, 133 MB (0.61).
// What is left is the way of each CTA to its first rows (loaded while the page
// table is looked at) and the barrier between its two passes: rows loaded ahead
// for the next head (128 registers, 4 CTAs) gained nothing over more CTAs.
//
// Read. One CTA per 16 or 32 packed rows and some heads, K or V; a thread's
// 16-byte stores cover neighbouring elements of a row.

#include "apr_internal.h"
#include "host_common.h"
#include "kv8.cuh"

namespace apr {
namespace {

constexpr int A_THREADS = 128;
// On an SM (96 registers; the three shapes above with 4 / 6 / 7: 24.0 / 24.2 / 24.9, 36.5 / 37.8 / 40.0,
// 30.1 / 31.6 / 33.5 us).
constexpr int A_CTAS = 5;
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

template <typename T, int D>
__global__ void __launch_bounds__(A_THREADS, A_CTAS) kv8_append_kernel(const __grid_constant__ Kv8View v,
                                                               const T* __restrict__ k, const T* __restrict__ vv,
                                                               long long ld, int heads_a_cta) {
  grid_dependency_wait();
  grid_launch_dependents();
  // the CTAs of a page, K and V and all heads, are neighbours: the rows they read are
  const int parts = 2 * ((v.kv_heads + heads_a_cta - 1) / heads_a_cta);
  const int unit = (int)(blockIdx.x / parts), part = (int)(blockIdx.x % parts);
  constexpr int HELD = 16 / sizeof(T);  // vectors of 8 values a thread keeps between the passes, 32 registers
  constexpr int ROW = D / 8;            // vectors of a row
  __shared__ float s_max[3][A_WARPS];
  const bool is_v = part & 1;
  const int g0 = (part >> 1) * heads_a_cta, g1 = min(g0 + heads_a_cta, v.kv_heads);

  // ---- which page: the slot-th that the sequence's rows go to, if it has so many
  int b = unit, slot = 0;
  if (v.row_start) {
    b = kv8_last_sequence(v, [&](int i) { return first_append_unit(v, i) <= unit; });
    slot = unit - first_append_unit(v, b);
    // every length and range is looked at, also one that no unit is found by
    if (part == 0 && unit < v.num_seqs && threadIdx.x == 0) kv8_len(v, unit), kv8_rows(v, unit);
  }
  const int len = kv8_len(v, b);
  const Kv8Span span = kv8_rows(v, b);
  const int first = len - span.n;  // position of row r0; rows of negative positions are skipped
  const int index = (max(first, 0) >> v.page_shift) + slot;
  if (slot < 0 || span.n == 0 || len == 0 || index > (len - 1) >> v.page_shift) return;
  const int page = v.table[(size_t)b * v.table_ld + index];  // (looked at when the first rows are on their way)

  const int page0 = index << v.page_shift;
  const int lo = max(max(first, 0), page0), hi = min(len, page0 + (1 << v.page_shift));
  const int held = lo - page0;
  const int nvec = (hi - lo) * ROW;
  // this thread's vectors: column (threadIdx.x % ROW), every (A_THREADS / ROW)-th row
  const long long step = ld * (A_THREADS / ROW);
  const T* src = (is_v ? vv : k) + (long long)(span.r0 + lo - first + (int)threadIdx.x / ROW) * ld +
                 (int)threadIdx.x % ROW * 8;
  src += (size_t)g0 * D;
  Vec8<T> keep[HELD];
  auto load = [&] {
#pragma unroll
    for (int j = 0; j < HELD; ++j)
      if ((int)threadIdx.x + j * A_THREADS < nvec) keep[j] = load8(src + j * step);
  };
  load();
  if (page < 0 || page >= v.num_pages) {
    if (threadIdx.x == 0) kv8_flag(v);
    return;
  }
  int8_t* codes = (is_v ? v.V : v.K) + kv8_codes_at(v, page, g0);
  float* scale = (is_v ? v.v_scale : v.k_scale) + kv8_scale_at(v, page, g0);
  for (int g = g0;; codes += (size_t)D << v.page_shift, ++scale) {
    const float s_old = held > 0 ? *scale : 0.f;
    // ---- the largest magnitude
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < HELD; ++j)
      if ((int)threadIdx.x + j * A_THREADS < nvec) m = amax_of(keep[j], m);
#pragma unroll 4
    for (int i = HELD; (int)threadIdx.x + i * A_THREADS < nvec; ++i) m = amax_of(load8(src + i * step), m);
    m = block_max<A_WARPS>(m, s_max[g & 1]);  // (the next head writes the other: one barrier a head)
    if (m > FLT_MAX) {                        // an infinity among them, for the whole CTA
      m = 0.f;
#pragma unroll
      for (int j = 0; j < HELD; ++j)
        if ((int)threadIdx.x + j * A_THREADS < nvec) m = finite_amax_of<T>(keep[j], m);
      for (int i = HELD; (int)threadIdx.x + i * A_THREADS < nvec; ++i) m = finite_amax_of<T>(load8(src + i * step), m);
      __syncthreads();
      m = block_max<A_WARPS>(m, s_max[2]);
    }

    // ---- the scale, and what the page held under a raised one
    const Kv8Scale s = kv8_rounding_to(fmaxf(s_old, kv8_scale_of(m)));
    if (threadIdx.x == 0 && (held == 0 || s.s > s_old)) *scale = s.s;
    if (held > 0 && s.s > s_old) {
      uint4* old = reinterpret_cast<uint4*>(codes);
      for (int i = threadIdx.x; i < held * D / 16; i += A_THREADS) {
        const uint4 w = old[i];
        uint4 y = kv8_requantise16(w, s_old, s);
        // (a code of -128 may have come from elsewhere)
        y.x = __vmaxs4(y.x, 0x81818181u), y.y = __vmaxs4(y.y, 0x81818181u);
        y.z = __vmaxs4(y.z, 0x81818181u), y.w = __vmaxs4(y.w, 0x81818181u);
        old[i] = y;
      }
    }

    // ---- the new codes
    uint2* dst = reinterpret_cast<uint2*>(codes + (size_t)held * D) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < HELD; ++j)
      if ((int)threadIdx.x + j * A_THREADS < nvec) dst[j * A_THREADS] = codes_of<T>(keep[j], s);
#pragma unroll 2
    for (int i = HELD; (int)threadIdx.x + i * A_THREADS < nvec; ++i)
      dst[i * A_THREADS] = codes_of<T>(load8(src + i * step), s);
    if (++g == g1) break;
    src += D;
    load();
  }
}

// ---------------------------------------------------------------- read
constexpr int R_THREADS = 256;

// R_ROWS: packed rows of a CTA.
template <typename T, int D, int R_ROWS>
__global__ void __launch_bounds__(R_THREADS) kv8_read_kernel(const __grid_constant__ Kv8View v, T* __restrict__ k,
                                                             T* __restrict__ vv, long long ld, int heads_a_cta) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int N = 16 / sizeof(T);             // values of a 16-byte store
  constexpr int ROW = D / N;                    // stores of a row
  constexpr int STEP = R_THREADS / ROW;         // rows between a thread's stores
  constexpr int EACH = (R_ROWS + STEP - 1) / STEP;
  __shared__ const int8_t* s_codes[R_ROWS];     // a row's codes of head g0; nullptr: none
  __shared__ const float* s_scale[R_ROWS];
  __shared__ int s_zero[R_ROWS];                // a row before its sequence's start
  const int parts = 2 * ((v.kv_heads + heads_a_cta - 1) / heads_a_cta), part = (int)(blockIdx.x % parts);
  const int row0 = (int)(blockIdx.x / parts) * R_ROWS;
  const bool is_v = part & 1;
  const int g0 = (part >> 1) * heads_a_cta, g1 = min(g0 + heads_a_cta, v.kv_heads);
  if (blockIdx.x == 0 && v.row_start)  // every range is looked at, also one that no row is found by
    for (int b = threadIdx.x; b < v.num_seqs; b += R_THREADS) kv8_rows(v, b);
  if (threadIdx.x < R_ROWS) {
    const int row = row0 + (int)threadIdx.x;
    int b = row;
    if (v.row_start) {  // the last sequence that begins at the row or before it
      int end = v.num_seqs;
      b = 0;
      while (end - b > 1) {
        const int mid = (b + end) / 2;
        if (v.row_start[mid] <= row)
          b = mid;
        else
          end = mid;
      }
    }
    const int8_t* codes = nullptr;
    const float* scale = nullptr;
    bool zero = false;
    if (row < v.num_rows) {
      const Kv8Span span = kv8_rows(v, b);
      if (row >= span.r0 && row < span.r0 + span.n) {
        const int pos = kv8_len(v, b) - span.n + (row - span.r0);  // negative: before the sequence's start
        const int page = pos < 0 ? -1 : kv8_page(v, b, pos >> v.page_shift);
        zero = pos < 0;
        if (page >= 0) {
          codes = (is_v ? v.V : v.K) + kv8_codes_at(v, page, g0) + (size_t)(pos & ((1 << v.page_shift) - 1)) * D;
          scale = (is_v ? v.v_scale : v.k_scale) + kv8_scale_at(v, page, g0);
        }
      }
    }
    s_codes[threadIdx.x] = codes;
    s_scale[threadIdx.x] = scale;
    s_zero[threadIdx.x] = zero;
  }
  __syncthreads();
  const int col = (int)threadIdx.x % ROW * N, r0 = (int)threadIdx.x / ROW;
  T* out = (is_v ? vv : k) + (long long)(row0 + r0) * ld + (size_t)g0 * D + col;
  const int8_t* from[EACH];
  const float* scale[EACH];
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int r = r0 + j * STEP;
    from[j] = r < R_ROWS && s_codes[r] ? s_codes[r] + col : nullptr;
    scale[j] = from[j] ? s_scale[r] : nullptr;
    if (r < R_ROWS && s_zero[r])
      for (int g = 0; g < g1 - g0; ++g)
        *reinterpret_cast<uint4*>(out + (long long)j * STEP * ld + (size_t)g * D) = make_uint4(0, 0, 0, 0);
  }
  const size_t head = (size_t)D << v.page_shift;
#pragma unroll 2
  for (int g = 0; g < g1 - g0; ++g, out += D) {
    uint2 w[EACH];
    float s[EACH];
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      w[j] = make_uint2(0, 0);
      s[j] = 0.f;
      if (from[j]) {
        if (N == 4)
          w[j].x = *reinterpret_cast<const uint32_t*>(from[j] + g * head);
        else
          w[j] = *reinterpret_cast<const uint2*>(from[j] + g * head);
        s[j] = scale[j][g];
      }
    }
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      if (!from[j]) continue;
      const uint32_t words[2] = {w[j].x ^ 0x80808080u, w[j].y ^ 0x80808080u};
      float2 x[4];
#pragma unroll
      for (int t = 0; t < N / 2; ++t)
        x[t] = __fmul2_rn(kv8_bytes_f32(words[t / 2], t % 2 * 2), make_float2(s[j], s[j]));
      uint4 y;
      if constexpr (N == 4)
        y = make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
      else
        y = make_uint4(pack2<T>(x[0].x, x[0].y), pack2<T>(x[1].x, x[1].y), pack2<T>(x[2].x, x[2].y),
                       pack2<T>(x[3].x, x[3].y));
      *reinterpret_cast<uint4*>(out + (long long)j * STEP * ld) = y;
    }
  }
}

// Heads of a CTA: all, or as few as it takes to give every SM `most` CTAs.
int heads_a_cta(long long units, int kv_heads, int most) {
  const long long want = (long long)most * num_sms() / (2 * units > 0 ? 2 * units : 1);  // CTAs of a unit, K or V
  return want <= 1 ? kv_heads : (int)(want >= kv_heads ? 1 : (kv_heads + want - 1) / want);
}

template <typename T, int D>
cudaError_t append_shape(const Kv8View& v, const void* k, const void* vv, long long ld, cudaStream_t s) {
  // the most pages that the rows can touch (first_append_unit)
  const long long pages = v.row_start ? (v.num_rows >> v.page_shift) + 2ll * v.num_seqs : v.num_seqs;
  const int heads = heads_a_cta(pages, v.kv_heads, 12);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pages * 2 * ((v.kv_heads + heads - 1) / heads)));
  cfg.blockDim = dim3(A_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_append_kernel<T, D>, v, (const T*)k, (const T*)vv, ld, heads);
}

template <typename T, int D, int R_ROWS>
cudaError_t launch_read(const Kv8View& v, void* k, void* vv, long long ld, cudaStream_t s) {
  const long long units = (v.num_rows + R_ROWS - 1) / R_ROWS;
  const int heads = heads_a_cta(units, v.kv_heads, 4);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * 2 * ((v.kv_heads + heads - 1) / heads)));
  cfg.blockDim = dim3(R_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_read_kernel<T, D, R_ROWS>, v, (T*)k, (T*)vv, ld, heads);
}

// 16 rows a CTA where 32 would leave an SM few CTAs, whose start and end then
// show (6007 float32 rows of 4 heads of 256: 10.4 us, 13.7 with 32); 32 where
// there are many (33700 bf16 rows of 8 of 128: 37 us, 39 with 16).
template <typename T, int D>
cudaError_t read_shape(const Kv8View& v, void* k, void* vv, long long ld, cudaStream_t s) {
  return v.num_rows < 32 * 3 * num_sms() / 2 ? launch_read<T, D, 16>(v, k, vv, ld, s) : launch_read<T, D, 32>(v, k, vv, ld, s);
}

template <typename T>
cudaError_t append_typed(const Kv8View& v, const void* k, const void* vv, long long ld, cudaStream_t s) {
  return v.dim == 64 ? append_shape<T, 64>(v, k, vv, ld, s)
                     : (v.dim == 128 ? append_shape<T, 128>(v, k, vv, ld, s) : append_shape<T, 256>(v, k, vv, ld, s));
}
template <typename T>
cudaError_t read_typed(const Kv8View& v, void* k, void* vv, long long ld, cudaStream_t s) {
  return v.dim == 64 ? read_shape<T, 64>(v, k, vv, ld, s)
                     : (v.dim == 128 ? read_shape<T, 128>(v, k, vv, ld, s) : read_shape<T, 256>(v, k, vv, ld, s));
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
