// The rotations' table and rows (include/apr_rope.h).

#include "apr_internal.h"
#include "host_common.h"
#include "rope.cuh"

namespace apr {
namespace {

// ---------------------------------------------------------------- the table
// Bound by memory, 8 bytes an entry written once, if an entry takes few instructions: this chip has
// two FP64 lanes an SM for 128 of FP32, so a 64-bit cosine of each entry takes 50 times as long as its
// store (400003 positions of 128 pairs: 2.9 ms). So a CTA has 32 columns (a pair, and TB_ROWS runs of positions one after the
// other, a run for each warp), takes cosine and sine in 64 bits for a column's first position, for one position and for
// a run, and turns on from there: a warp by whole runs to its own, then by one position at a time, each a
// complex product of numbers of two float32 (rope.cuh), cosine and sine in the two halves of packed instructions: 20 an entry.
// A product and its factor are off by some 2^-46, a run of 64 by 2^-40 at the most, far below half a step of the float32 result.
// 400003 positions of 128 pairs 76 us, 0.81 of the HBM rate (runs of 32 91, of 128 73; 64-bit evaluations for every run 108); 8192 of 32
// pairs 3.6 us (8.1).
constexpr int TB_ROWS = 8, TB_THREADS = 32 * TB_ROWS;
constexpr int TB_RUN = 64;

struct Point {
  double c, s;
};
// Cosine and sine of n f (1 / 2 pi in two doubles takes the whole turns off; Taylor's series up to pi / 4, the
// first term left out below 2^-53).
__device__ __forceinline__ Point point_of(double n, double f) {
  constexpr double C0 = 0.15915494309189535, C1 = -9.839338337591243e-18;  // 1 / (2 pi)
  const double p = n * f, pe = fma(n, f, -p);
  const double t = p * C0, te = fma(p, C0, -t) + (p * C1 + pe * C0);
  const double whole = rint(t);
  double r = (t - whole) + te;                      // turns, within a half
  const double q = rint(4.0 * r);
  const double x = (r - 0.25 * q) * 6.283185307179586, z = x * x;
  double s = fma(z, -1.0 / 1307674368000.0, 1.0 / 6227020800.0);
  s = fma(z, s, -1.0 / 39916800.0);
  s = fma(z, s, 1.0 / 362880.0);
  s = fma(z, s, -1.0 / 5040.0);
  s = fma(z, s, 1.0 / 120.0);
  s = fma(z, s, -1.0 / 6.0);
  s = fma(z * x, s, x);
  double c = fma(z, 1.0 / 20922789888000.0, -1.0 / 87178291200.0);
  c = fma(z, c, 1.0 / 479001600.0);
  c = fma(z, c, -1.0 / 3628800.0);
  c = fma(z, c, 1.0 / 40320.0);
  c = fma(z, c, -1.0 / 720.0);
  c = fma(z, c, 1.0 / 24.0);
  c = fma(z, c, -0.5);
  c = fma(z, c, 1.0);
  const int k = (int)q & 3;
  return Point{k == 0 ? c : (k == 1 ? -s : (k == 2 ? -c : s)), k == 0 ? s : (k == 1 ? c : (k == 2 ? -s : -c))};
}

__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// (cosine, sine) of an angle, each in two float32.
struct Turn {
  float2 hi, lo;
};
// z turned by w: (c, s) w.c + (-s, c) w.s.
__device__ __forceinline__ Turn turned(const Turn& z, const Turn& w) {
  const float2 a_hi = make_float2(w.hi.x, w.hi.x), a_lo = make_float2(w.lo.x, w.lo.x);
  const float2 b_hi = make_float2(w.hi.y, w.hi.y), b_lo = make_float2(w.lo.y, w.lo.y);
  const float2 xh = make_float2(-z.hi.y, z.hi.x), xl = make_float2(-z.lo.y, z.lo.x);
  const float2 u = __fmul2_rn(z.hi, a_hi), v = __fmul2_rn(xh, b_hi);
  const float2 ue = __ffma2_rn(z.lo, a_hi, __ffma2_rn(z.hi, a_lo, __ffma2_rn(z.hi, a_hi, neg2(u))));
  const float2 ve = __ffma2_rn(xl, b_hi, __ffma2_rn(xh, b_lo, __ffma2_rn(xh, b_hi, neg2(v))));
  const float2 t = __fadd2_rn(u, v), d = __fadd2_rn(t, neg2(u));
  const float2 e = __fadd2_rn(__fadd2_rn(u, neg2(__fadd2_rn(t, neg2(d)))), __fadd2_rn(v, neg2(d)));
  const float2 r = __fadd2_rn(e, __fadd2_rn(ue, ve));
  Turn y;
  y.hi = __fadd2_rn(t, r);
  y.lo = __fadd2_rn(r, neg2(__fadd2_rn(y.hi, neg2(t))));
  return y;
}

__global__ void __launch_bounds__(TB_THREADS) rope_table_kernel(const float* __restrict__ inv_freq, unsigned pairs,
                                                                long long first, long long positions, double scale,
                                                                int run, unsigned columns, float2* __restrict__ table) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ Turn s_turn[3][32];  // the first position of a column, one position, a run
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const unsigned column = min(blockIdx.x * 32 + lane, columns - 1), pair = column % pairs;
  const long long begin = (long long)(column / pairs) * (TB_ROWS * run);
  if (row < 3) {
    const Point z = point_of(row == 0 ? (double)(first + begin) : (row == 1 ? 1.0 : (double)run), (double)inv_freq[pair]);
    const double by = row == 0 ? scale : 1.0, c = z.c * by, s = z.s * by;
    const float2 hi = make_float2((float)c, (float)s);
    s_turn[row][lane] = Turn{hi, make_float2((float)(c - (double)hi.x), (float)(s - (double)hi.y))};
  }
  __syncthreads();
  const long long p0 = begin + row * run;
  if (blockIdx.x * 32 + lane >= columns || p0 >= positions) return;
  Turn z = s_turn[0][lane];
  const Turn one = s_turn[1][lane], whole = s_turn[2][lane];
  for (int i = 0; i < row; ++i) z = turned(z, whole);
  float2* to = table + p0 * pairs + pair;
  const int n = (int)min((long long)run, positions - p0);
  *to = z.hi;
#pragma unroll 4
  for (int k = 1; k < n; ++k) {
    to += pairs;
    z = turned(z, one);
    *to = z.hi;
  }
}

// ---------------------------------------------------------------- rows
// A row read and written once, its turns read once for all its heads: bound by memory. Where there is a norm, by its latency: a warp
// loads its next heads when the last ones are stored, at 24 warps an SM (78 registers: every step is rounded by itself and a mean of squares has
// 45 bits, rope.cuh). 16390 normed bf16 rows of 32 heads of 128 on three axes take 61 us, 0.68 of the HBM rate with 62 % of the issue
// slots taken, loads the largest stall; 8192 float32 rows of 16 heads of 256 51 us, 0.79; 5329 fp16 rows of 16 heads of 72 9.4 us (9 of 16
// lanes have a unit); one row 3 us.
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
  constexpr int GROUPS = RR_THREADS / LANES;
  a.heads_a_group = rope_heads_a_group(a.num_rows, a.heads, GROUPS * 8ll * num_sms());
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
  // runs as long as they may be that give every SM two CTAs
  int run = TB_RUN;
  while (run > 8 && positions * pairs < 2ll * TB_THREADS * run * num_sms()) run /= 2;
  const long long spans = (positions + TB_ROWS * run - 1) / (TB_ROWS * run), columns = spans * pairs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((columns + 31) / 32));
  cfg.blockDim = dim3(TB_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_table_kernel, inv_freq, (unsigned)pairs, first, positions, scale, run, (unsigned)columns,
                            (float2*)table);
}

cudaError_t launch_rope_rows(const RopeView& r, const RopeRows& a, int type, cudaStream_t s) {
  if (type == APR_T_F32) return rows_typed<float>(r, a, s);
  if (type == APR_T_F16) return rows_typed<__half>(r, a, s);
  return rows_typed<__nv_bfloat16>(r, a, s);
}

}  // namespace apr
