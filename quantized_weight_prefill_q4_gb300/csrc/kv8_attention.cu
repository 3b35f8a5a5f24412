// Attention of a sequence's last rows over its 8-bit paged KV cache
// (include/apr_kv8.h):
//   p_j = softmax_j(scale q . (c_j s)),  out = sum_j p_j (c'_j s'),  w_j = sum of p_j
//
// Work. The (row, head) pairs of a sequence that read the same KV head are
// taken PAIRS at a time; one such group of pairs over all the sequence's
// positions is a segment, and its positions go in units of UNIT. The units of
// all segments are numbered through, and each CTA takes an equal, contiguous
// share of them, so that sequences of any lengths in one batch keep every SM
// equally busy. A segment within one CTA's share is finished there; otherwise
// each CTA that has a piece of it writes the piece's unnormalised sums with
// their reference maximum and total, and a second kernel combines the pieces in
// order. A third kernel, where the weights are wanted, turns the scores that
// the first one kept into them once the totals are known.
//
// The softmax works in base 2.

#include "apr_internal.h"
#include "host_common.h"
#include "kv8.cuh"

namespace apr {
namespace {

constexpr int THREADS = 256;
constexpr int UNIT = 64;   // positions of a unit of work
constexpr int PAIRS = 8;   // (row, head) pairs of a segment

struct AttnArgs {
  Kv8View v;
  const void* q;
  void* out;
  long long ldq, ldo;
  int type, heads, group;
  float scale_log2;  // softmax scale times log2(e)
  int ctas;          // of the grid; no more than there are units share them
  int* prefix;       // [num_seqs + 1] first unit of each sequence (written by CTA 0)
  float2* part_ml;   // [2 ctas][PAIRS] reference maximum and total of a piece
  float* part_o;     // [2 ctas][PAIRS][dim]
  float2* final_ml;  // [rows][heads] maximum and 1 / total, or nullptr
  float* scores;     // [rows][heads][max_len] scores in base 2, or nullptr
  float* weights;
  long long weights_ld;
  int accumulate;
};

__device__ __forceinline__ float load_any(const void* p, int type, size_t i) {
  if (type == APR_T_F32) return static_cast<const float*>(p)[i];
  if (type == APR_T_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int type, size_t i, float x) {
  if (type == APR_T_F32)
    static_cast<float*>(p)[i] = x;
  else if (type == APR_T_F16)
    static_cast<__half*>(p)[i] = __float2half_rn(x);
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}

// Units of one segment of a sequence, and its segments.
__device__ __forceinline__ int segment_units(int len) { return max(1, (len + UNIT - 1) / UNIT); }
__device__ __forceinline__ int segment_count(const AttnArgs& a, int n) {
  return (n * a.group + PAIRS - 1) / PAIRS * a.v.kv_heads;
}
__device__ __forceinline__ int sequence_units(const AttnArgs& a, int b) {
  const int n = kv8_rows(a.v, b).n;
  return n == 0 ? 0 : segment_count(a, n) * segment_units(kv8_len(a.v, b));
}

// The `ctas` CTAs that share `total` units: each has one at least. CTA c has the units first_unit(c) .. first_unit(c + 1) - 1 of `total`; the
// CTA that has unit u.
__device__ __forceinline__ int first_unit(int c, int ctas, int total) {
  return (int)((long long)c * total / ctas);
}
__device__ __forceinline__ int cta_of(int u, int ctas, int total) {
  return (int)((((long long)u + 1) * ctas - 1) / total);
}

template <int D>
__global__ void __launch_bounds__(THREADS) kv8_attention_kernel(const AttnArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  constexpr int TILE = 32;
  __shared__ float sq[PAIRS][D];
  __shared__ float sk[TILE][D + 1];
  __shared__ float sp[PAIRS][TILE];
  __shared__ int s_scan[THREADS / 32];
  __shared__ int s_find[3];
  const Kv8View& v = a.v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // ---- the units of the sequences, and where this CTA's share begins
  int total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int base = 0;
    const int u0 = pass ? first_unit(blockIdx.x, min(a.ctas, total), total) : 0;
    for (int b0 = 0; b0 < v.num_seqs; b0 += THREADS) {
      const int b = b0 + (int)threadIdx.x;
      const int n = b < v.num_seqs ? sequence_units(a, b) : 0;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = inc;
      __syncthreads();
      int before = base, all = 0;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += s_scan[w];
        all += s_scan[w];
      }
      const int at = before + inc - n;
      if (pass && n > 0 && at <= u0 && u0 < at + n) {
        s_find[0] = b;
        s_find[1] = at;
      }
      if (pass && blockIdx.x == 0 && b < v.num_seqs) a.prefix[b] = at;
      base += all;
    }
    total = base;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.prefix[v.num_seqs] = total;
  __syncthreads();
  const int ctas = min(a.ctas, total);
  if ((int)blockIdx.x >= ctas) return;
  int u = first_unit(blockIdx.x, ctas, total);
  const int u_begin = u, u_end = first_unit(blockIdx.x + 1, ctas, total);
  int b = s_find[0], seq_u0 = s_find[1];

  while (u < u_end) {
    const int len = kv8_len(v, b);
    const Kv8Span span = kv8_rows(v, b);
    const int su = segment_units(len), nseg = span.n ? segment_count(a, span.n) : 0;
    if (u >= seq_u0 + nseg * su) {  // the next sequence that has rows
      seq_u0 += nseg * su;
      ++b;
      continue;
    }
    const int seg = (u - seq_u0) / su, seg_u0 = seq_u0 + seg * su;
    const int g = seg % v.kv_heads, p0 = seg / v.kv_heads * PAIRS, np = min(PAIRS, span.n * a.group - p0);
    const int ue = min(u_end, seg_u0 + su);
    const int k0 = (u - seg_u0) * UNIT, k1 = min(len, (ue - seg_u0) * UNIT);
    // ---- the pairs' query rows
    __syncthreads();
    for (int i = threadIdx.x; i < PAIRS * D; i += THREADS) {
      const int p = i / D, c = i % D, pair = p0 + p;
      const int row = span.r0 + pair / a.group, head = g * a.group + pair % a.group;
      sq[p][c] = p < np ? load_any(a.q, a.type, (size_t)row * a.ldq + (size_t)head * D + c) : 0.f;
    }
    const int pair = p0 + warp;  // this warp's pair
    const bool live = warp < np;
    const int row = span.r0 + pair / a.group, head = g * a.group + pair % a.group;
    const int limit = len - span.n + pair / a.group + 1;  // positions the pair sees
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
    for (int k = k0; k < k1; k += TILE) {
      const int page = kv8_page(v, b, k >> v.page_shift);
      const size_t at = page < 0 ? 0 : kv8_codes_at(v, page, g) + (size_t)(k & ((1 << v.page_shift) - 1)) * D;
      const float ks = page < 0 ? 0.f : v.k_scale[kv8_scale_at(v, page, g)];
      const float vs = page < 0 ? 0.f : v.v_scale[kv8_scale_at(v, page, g)];
      __syncthreads();
      for (int i = threadIdx.x; i < TILE * D / 4; i += THREADS) {
        const uint32_t w = page < 0 ? 0 : reinterpret_cast<const uint32_t*>(v.K + at)[i];
#pragma unroll
        for (int t = 0; t < 4; ++t) sk[4 * i / D][4 * i % D + t] = (float)kv8_byte(w, t);
      }
      __syncthreads();
      float s = -INFINITY;
      if (live && k + lane < min(limit, len) && page >= 0) {
        s = 0.f;
        for (int c = 0; c < D; ++c) s = fmaf(sq[warp][c], sk[lane][c], s);
        s *= ks * a.scale_log2;
      }
      if (live && a.scores && k + lane < len) a.scores[((size_t)row * a.heads + head) * v.max_len + k + lane] = s;
      float top = s;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float m_new = fmaxf(m, top), ref = m_new == -INFINITY ? 0.f : m_new;
      const float f = exp2f(m - ref), p = exp2f(s - ref);
      m = m_new;
      l = l * f + p;  // per lane
      sp[warp][lane] = p * vs;
      __syncthreads();
      for (int i = threadIdx.x; i < TILE * D / 4; i += THREADS) {
        const uint32_t w = page < 0 ? 0 : reinterpret_cast<const uint32_t*>(v.V + at)[i];
#pragma unroll
        for (int t = 0; t < 4; ++t) sk[4 * i / D][4 * i % D + t] = (float)kv8_byte(w, t);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float acc = o[i] * f;
        for (int j = 0; j < TILE; ++j) acc = fmaf(sp[warp][j], sk[j][32 * i + lane], acc);
        o[i] = acc;
      }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (m == -INFINITY) m = 0.f;
    const bool whole = u == seg_u0 && ue == seg_u0 + su;
    if (live && whole) {
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        store_any(a.out, a.type, (size_t)row * a.ldo + (size_t)head * D + 32 * i + lane, o[i] * inv);
      if (a.final_ml && lane == 0) a.final_ml[(size_t)row * a.heads + head] = make_float2(m, inv);
    } else if (live) {
      const size_t slot = (size_t)(2 * blockIdx.x + (u_begin > seg_u0 ? 0 : 1)) * PAIRS + warp;
      if (lane == 0) a.part_ml[slot] = make_float2(m, l);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) a.part_o[slot * D + 32 * i + lane] = o[i];
    }
    u = ue;
  }
}

// The pieces of each segment that more than one CTA had: a warp for each
// (row, head), pieces in order.
template <int D>
__global__ void __launch_bounds__(256) kv8_combine_kernel(const AttnArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const Kv8View& v = a.v;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const Kv8Span span = kv8_rows(v, b);
  const int id = (int)blockIdx.x * 8 + ((int)threadIdx.x >> 5);  // pair * kv_heads + g
  const int g = id % v.kv_heads, pair = id / v.kv_heads;
  if (pair >= span.n * a.group) return;
  const int total = a.prefix[v.num_seqs], ctas = min(a.ctas, total), su = segment_units(kv8_len(v, b));
  const int u0 = a.prefix[b] + (pair / PAIRS * v.kv_heads + g) * su;
  const int c0 = cta_of(u0, ctas, total), c1 = cta_of(u0 + su - 1, ctas, total);
  if (c0 == c1) return;
  // the first CTA wrote it as the segment it began, the others as the one they continued
  auto slot = [&](int c) { return (size_t)(c == c0 ? 2 * c + 1 : 2 * c) * PAIRS + pair % PAIRS; };
  float m = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) {
    const float2 ml = a.part_ml[slot(c)];
    if (ml.y > 0.f) m = fmaxf(m, ml.x);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  if (m == -INFINITY) m = 0.f;
  float l = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float2 ml = a.part_ml[slot(c)];
    const float f = ml.y > 0.f || ml.y != ml.y ? exp2f(ml.x - m) : 0.f;
    l = fmaf(f, ml.y, l);
    const float* po = a.part_o + slot(c) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = fmaf(f, po[32 * i + lane], o[i]);
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  const int row = span.r0 + pair / a.group, head = g * a.group + pair % a.group;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    store_any(a.out, a.type, (size_t)row * a.ldo + (size_t)head * D + 32 * i + lane, o[i] * inv);
  if (a.final_ml && lane == 0) a.final_ml[(size_t)row * a.heads + head] = make_float2(m, inv);
}

// w_j: a thread for each position of a sequence and KV head, its pairs in order.
__global__ void __launch_bounds__(256) kv8_weights_kernel(const AttnArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const Kv8View& v = a.v;
  const int g = blockIdx.y, b = blockIdx.z;
  const long long j = (long long)blockIdx.x * 256 + threadIdx.x;
  const int len = kv8_len(v, b);
  const Kv8Span span = kv8_rows(v, b);
  if (j >= a.weights_ld || (a.accumulate && j >= len)) return;
  float* w = a.weights + ((size_t)b * v.kv_heads + g) * a.weights_ld + j;
  float sum = 0.f;
  if (j < len) {
    for (int i = 0; i < span.n; ++i)
#pragma unroll 4
      for (int h = 0; h < a.group; ++h) {
        const size_t at = (size_t)(span.r0 + i) * a.heads + g * a.group + h;
        const float2 ml = a.final_ml[at];
        sum += exp2f(a.scores[at * v.max_len + j] - ml.x) * ml.y;
      }
    if (a.accumulate && j < len - span.n) sum += *w;
  }
  *w = sum;
}

struct Layout {
  int ctas;
  size_t prefix, part_ml, part_o, final_ml, scores, bytes;
};

Layout layout_of(const Kv8View& v, const Kv8Attention& a) {
  Layout l;
  const int group = a.heads / v.kv_heads;
  const long long segs = ((long long)v.num_rows * group / PAIRS + v.num_seqs) * v.kv_heads;  // at most
  const long long most = segs * (v.max_len / UNIT + 1);
  l.ctas = (int)(most < 2 * num_sms() ? (most < 1 ? 1 : most) : 2 * num_sms());
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
  };
  l.prefix = take(((size_t)v.num_seqs + 1) * 4);
  l.part_ml = take((size_t)2 * l.ctas * PAIRS * 8);
  l.part_o = take((size_t)2 * l.ctas * PAIRS * v.dim * 4);
  l.final_ml = take(a.weights ? (size_t)v.num_rows * a.heads * 8 : 0);
  l.scores = take(a.weights ? (size_t)v.num_rows * a.heads * v.max_len * 4 : 0);
  l.bytes = at;
  return l;
}

template <int D>
cudaError_t launch_dim(const AttnArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_attention_kernel<D>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(((long long)a.v.max_rows * a.heads + 7) / 8), (unsigned)a.v.num_seqs);
  cfg.blockDim = dim3(256);
  e = cudaLaunchKernelEx(&cfg, kv8_combine_kernel<D>, a);
  if (e != cudaSuccess || !a.weights) return e;
  const long long span = a.accumulate ? a.v.max_len : a.weights_ld;
  cfg.gridDim = dim3((unsigned)((span + 255) / 256), (unsigned)a.v.kv_heads, (unsigned)a.v.num_seqs);
  return cudaLaunchKernelEx(&cfg, kv8_weights_kernel, a);
}

}  // namespace

size_t kv8_attention_scratch(const Kv8View& v, const Kv8Attention& a) { return layout_of(v, a).bytes; }

cudaError_t launch_kv8_attention(const Kv8View& v, const Kv8Attention& in, void* scratch, cudaStream_t s) {
  const Layout l = layout_of(v, in);
  uint8_t* base = static_cast<uint8_t*>(scratch);
  AttnArgs a = {};
  a.v = v;
  a.q = in.q;
  a.out = in.out;
  a.ldq = in.ldq;
  a.ldo = in.ldo;
  a.type = in.type;
  a.heads = in.heads;
  a.group = in.heads / v.kv_heads;
  a.scale_log2 = in.scale * 1.4426950408889634f;
  a.ctas = l.ctas;
  a.prefix = reinterpret_cast<int*>(base + l.prefix);
  a.part_ml = reinterpret_cast<float2*>(base + l.part_ml);
  a.part_o = reinterpret_cast<float*>(base + l.part_o);
  if (in.weights) {
    a.final_ml = reinterpret_cast<float2*>(base + l.final_ml);
    a.scores = reinterpret_cast<float*>(base + l.scores);
    a.weights = in.weights;
    a.weights_ld = in.weights_ld;
    a.accumulate = in.accumulate;
  }
  if (v.dim == 64) return launch_dim<64>(a, s);
  if (v.dim == 128) return launch_dim<128>(a, s);
  return launch_dim<256>(a, s);
}

}  // namespace apr
