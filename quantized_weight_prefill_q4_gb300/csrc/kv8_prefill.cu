// Attention of chunks of rows over their sequences' 8-bit paged KV caches
// (include/apr_kv8.h): for each (row, head) pair
//   p_j = softmax_j(scale q . (c_j s)),  out = sum_j p_j (c'_j s'),  j <= its position
//
// A warp a pair, 32 positions at a time: a lane has a position's score, then D / 32
// dims of the sum, one pass with the running maximum and sum. float32 throughout.

#include "apr_internal.h"
#include "host_common.h"
#include "kv8.cuh"

namespace apr {
namespace {

constexpr int WARPS = 4;

struct PrefillArgs {
  Kv8View v;
  const void* q;
  void* out;
  long long ldq, ldo;
  int heads, group;
  float scale_log2;  // softmax scale times log2(e)
};

template <typename T>
__device__ __forceinline__ float value_at(const T* p) {
  if constexpr (sizeof(T) == 4) return *p;
  else return (float)*p;
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * WARPS) kv8_prefill_kernel(const __grid_constant__ PrefillArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ float s_q[WARPS][D];
  const Kv8View& v = a.v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0)  // every length and range is looked at, also one that no row is found by
    for (int b = threadIdx.x; b < v.num_seqs; b += 32 * WARPS) kv8_len(v, b), kv8_rows(v, b);
  const long long pair = (long long)blockIdx.x * WARPS + warp;
  if (pair >= (long long)v.num_rows * a.heads) return;
  const int row = (int)(pair / a.heads), h = (int)(pair % a.heads), g = h / a.group;
  const int b = kv8_sequence_of(v, row);
  const Kv8Span span = kv8_rows(v, b);
  if (row < span.r0 || row >= span.r0 + span.n) return;  // no sequence's row
  const int len = kv8_len(v, b), sees = min(len, len - span.n + row - span.r0 + 1);
  const T* q = static_cast<const T*>(a.q) + row * a.ldq + (size_t)h * D;
  bool odd = false;
  for (int d = lane; d < D; d += 32) {
    const float x = value_at(q + d);
    odd |= !(fabsf(x) <= FLT_MAX);
    s_q[warp][d] = x * a.scale_log2;
  }
  odd = __any_sync(0xffffffffu, odd);
  __syncwarp();
  constexpr int EACH = D / 32;
  float m = -INFINITY, l = 0.f, o[EACH] = {};
  for (int k0 = 0; k0 < sees; k0 += 32) {
    const int page = max(kv8_page(v, b, k0 >> v.page_shift), 0);
    const size_t codes = kv8_codes_at(v, page, g) + (size_t)(k0 & ((1 << v.page_shift) - 1)) * D;
    const float ks = v.k_scale[kv8_scale_at(v, page, g)], vs = v.v_scale[kv8_scale_at(v, page, g)];
    const char4* kc = reinterpret_cast<const char4*>(v.K + codes + (size_t)lane * D);
    float s = 0.f;
#pragma unroll 8
    for (int d = 0; d < D / 4; ++d) {
      const char4 c = kc[d];
      const float4 x = reinterpret_cast<const float4*>(s_q[warp])[d];
      s = fmaf(x.x, c.x, fmaf(x.y, c.y, fmaf(x.z, c.z, fmaf(x.w, c.w, s))));
    }
    s = k0 + lane < sees ? s * ks : -INFINITY;
    float top = s;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    const float m_new = fmaxf(m, top);
    const float f = exp2f(m - m_new), p = exp2f(s - m_new);
    float sum = p;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    l = l * f + sum;
    m = m_new;
#pragma unroll
    for (int e = 0; e < EACH; ++e) o[e] *= f;
    const float ps = p * (vs * 0x1p-24f);  // (sums of large values stay in range)
    for (int j = 0; j < 32; ++j) {
      const float w = __shfl_sync(0xffffffffu, ps, j);
#pragma unroll
      for (int e = 0; e < EACH; ++e) o[e] = fmaf(w, (float)v.V[codes + (size_t)j * D + lane + 32 * e], o[e]);
    }
  }
  T* out = static_cast<T*>(a.out) + row * a.ldo + (size_t)h * D;
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    float y = l > 0.f ? o[e] / l * 0x1p24f : 0.f;
    if (odd && sees > 0) y = __int_as_float(0x7fffffff);
    out[lane + 32 * e] = (T)y;
  }
}

template <typename T, int D>
cudaError_t launch_shape(const PrefillArgs& a, cudaStream_t s) {
  const long long pairs = (long long)a.v.num_rows * a.heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((pairs + WARPS - 1) / WARPS));
  cfg.blockDim = dim3(32 * WARPS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_prefill_kernel<T, D>, a);
}
template <typename T>
cudaError_t launch_typed(const PrefillArgs& a, cudaStream_t s) {
  return a.v.dim == 64 ? launch_shape<T, 64>(a, s) : (a.v.dim == 128 ? launch_shape<T, 128>(a, s) : launch_shape<T, 256>(a, s));
}

}  // namespace

size_t kv8_prefill_scratch(const Kv8View&, int, int) { return 0; }

cudaError_t launch_kv8_prefill(const Kv8View& v, int type, const void* q, long long ldq, void* out, long long ldo,
                               int heads, float scale, void*, cudaStream_t s) {
  const PrefillArgs a{v, q, out, ldq, ldo, heads, heads / v.kv_heads, scale * 1.4426950408889634f};
  if (type == APR_T_F32) return launch_typed<float>(a, s);
  if (type == APR_T_F16) return launch_typed<__half>(a, s);
  return launch_typed<__nv_bfloat16>(a, s);
}

}  // namespace apr
