// The rotations' table and rows (include/apr_rope.h).

#include "apr_internal.h"
#include "host_common.h"
#include "rope.cuh"

namespace apr {
namespace {

// ---------------------------------------------------------------- the table
constexpr int TB_THREADS = 256;

__global__ void __launch_bounds__(TB_THREADS) rope_table_kernel(const float* __restrict__ inv_freq, int pairs,
                                                                long long first, long long entries, double scale,
                                                                float2* __restrict__ table) {
  grid_dependency_wait();
  grid_launch_dependents();
  for (long long i = (long long)blockIdx.x * TB_THREADS + threadIdx.x; i < entries; i += (long long)gridDim.x * TB_THREADS) {
    const double angle = (double)(first + i / pairs) * (double)inv_freq[i % pairs];  // exact: 30 and 24 bits
    double s, c;
    sincos(angle, &s, &c);
    table[i] = make_float2((float)(c * scale), (float)(s * scale));
  }
}

// ---------------------------------------------------------------- rows
constexpr int RR_THREADS = 256;

template <typename T, int LANES, int EACH>
__global__ void __launch_bounds__(RR_THREADS) rope_rows_kernel(const __grid_constant__ RopeView r,
                                                               const __grid_constant__ RopeRows a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const long long group = (long long)blockIdx.x * (RR_THREADS / LANES) + threadIdx.x / LANES;
  rope_rows_group<T, LANES, EACH>(r, a, group, threadIdx.x % LANES, 0, true);
}

template <typename T, int LANES, int EACH>
cudaError_t rows_shape(const RopeView& r, RopeRows a, cudaStream_t s) {
  // heads of a group: as many as leave every SM some CTAs
  a.heads_a_group = a.heads;
  constexpr int GROUPS = RR_THREADS / LANES;
  while (a.heads_a_group > 1 &&
         (long long)a.num_rows * ((a.heads + a.heads_a_group - 1) / a.heads_a_group) < (long long)GROUPS * 8 * num_sms())
    a.heads_a_group = (a.heads_a_group + 1) / 2;
  const long long groups = (long long)a.num_rows * ((a.heads + a.heads_a_group - 1) / a.heads_a_group);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((groups + GROUPS - 1) / GROUPS));
  cfg.blockDim = dim3(RR_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_rows_kernel<T, LANES, EACH>, r, a);
}
template <typename T>
cudaError_t rows_typed(const RopeView& r, const RopeRows& a, cudaStream_t s) {
  if (a.dim <= 64) return rows_shape<T, 8, 1>(r, a, s);
  if (a.dim <= 128) return rows_shape<T, 16, 1>(r, a, s);
  if (a.dim <= 256) return rows_shape<T, 32, 1>(r, a, s);
  return rows_shape<T, 32, 2>(r, a, s);
}

}  // namespace

cudaError_t launch_rope_table(const float* inv_freq, int pairs, long long first, long long positions, double scale,
                              float* table, cudaStream_t s) {
  const long long entries = positions * pairs, blocks = (entries + TB_THREADS - 1) / TB_THREADS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < 16ll * num_sms() ? blocks : 16ll * num_sms()));
  cfg.blockDim = dim3(TB_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_table_kernel, inv_freq, pairs, first, entries, scale, (float2*)table);
}

cudaError_t launch_rope_rows(const RopeView& r, const RopeRows& a, int type, cudaStream_t s) {
  if (type == APR_T_F32) return rows_typed<float>(r, a, s);
  if (type == APR_T_F16) return rows_typed<__half>(r, a, s);
  return rows_typed<__nv_bfloat16>(r, a, s);
}

}  // namespace apr
