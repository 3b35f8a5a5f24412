// Eviction from the 8-bit paged KV cache (include/apr_kv8.h): which positions
// a sequence keeps, and their move into fresh pages.
//
// Selection. One cluster of CTAs per (sequence, KV head), each CTA a
// contiguous share of the positions. The weights are mapped to unsigned keys
// that order as the numbers do, and the key of the last one kept is found by
// three rounds of histograms over 11, 11 and 10 bits of it, each round's
// counts added up over the cluster through distributed shared memory. A second
// pass writes the kept positions in order: each CTA knows from its peers'
// counts how many it has before it, and takes the equal keys lowest position
// first. Every count is a whole number, so the result does not depend on the
// order of the atomics. The weights (4 bytes a position) are read five times,
// from DRAM once: they fit L2.
//
// Move. One CTA per (fresh page, KV head, K or V): the kept rows' codes are
// gathered once for the largest value, once (from L1) to be quantised anew.

#include "apr_internal.h"
#include "host_common.h"
#include "kv8.cuh"

namespace apr {
namespace {

constexpr int S_CTAS = 8;  // CTAs of a cluster, the portable size
constexpr int S_THREADS = 512;
constexpr int S_WARPS = S_THREADS / 32;
constexpr int S_BINS = 2048;

// Unsigned keys in the numbers' order: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, int rank) {
  uint32_t r;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(mapa_shared(smem_u32(p), (uint32_t)rank)) : "memory");
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  cluster_arrive();
  cluster_wait();
}

// Sum of x over the threads before this one, and over all of them (*total).
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < S_WARPS; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  __syncthreads();
  *total = all;
  return before + inc - x;
}

struct EvictArgs {
  const float* weights;
  long long weights_ld;
  int budget, recent, fresh_w;
  const int* fresh;
  int* table_out;
  int* lens_out;
  float* weights_out;
  long long weights_out_ld;
  int* kept;
};

__global__ void __launch_bounds__(S_THREADS) kv8_select_kernel(Kv8View v, EvictArgs a) {
  kv8_ready();
  grid_launch_dependents();  // of the move, which waits for this grid's end and lets nothing start before its own
  __shared__ uint32_t hist[S_BINS];
  __shared__ uint32_t chosen[2];  // the round's bin, and how many of it are kept
  __shared__ uint32_t counts[2];  // this CTA's keys above the border, and equal to it
  __shared__ int warp_sums[S_WARPS];
  const int rank = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int len = kv8_len(v, b);
  const size_t bg = (size_t)b * v.kv_heads + g;
  const float* w = a.weights + bg * a.weights_ld;
  float* wo = a.weights_out + bg * a.weights_out_ld;
  int* kept = a.kept + bg * a.budget;
  const int now = min(len, a.budget);
  const int all = S_CTAS * S_THREADS, tid = rank * S_THREADS + threadIdx.x;
  if (g == 0) {  // the sequence's table row and length
    const int pages = (now + (1 << v.page_shift) - 1) >> v.page_shift;
    const int* own = v.table + (size_t)b * v.table_ld;
    for (int i = tid; i < v.table_ld; i += all)
      a.table_out[(size_t)b * v.table_ld + i] =
          i >= pages ? -1 : (len > a.budget ? a.fresh[(size_t)b * a.fresh_w + i] : own[i]);
    if (tid == 0) a.lens_out[b] = now;
  }
  for (long long j = now + tid; j < a.weights_out_ld; j += all) wo[j] = 0.f;
  for (int j = now + tid; j < a.budget; j += all) kept[j] = -1;
  if (len <= a.budget) {  // the whole cluster: nothing to cut
    for (int j = tid; j < len; j += all) {
      wo[j] = w[j];
      kept[j] = j;
    }
    return;
  }
  const int old = len - a.recent;            // positions that compete
  const int need = a.budget - a.recent;      // of them, how many are kept (< old)
  for (int j = tid; j < a.recent; j += all) {
    wo[need + j] = w[old + j];
    kept[need + j] = old + j;
  }
  if (need == 0) return;
  const int share = ((old + S_CTAS - 1) / S_CTAS + 3) & ~3;
  const int lo = min(rank * share, old), hi = min(lo + share, old);

  // ---- the key of the last position kept: border, of whose equals `take` are kept
  uint32_t border = 0, take = (uint32_t)need;
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int bits = round == 2 ? 10 : 11, shift = round == 0 ? 21 : (round == 1 ? 10 : 0);
    for (int i = threadIdx.x; i < S_BINS; i += S_THREADS) hist[i] = 0;
    __syncthreads();
    const uint32_t above = round == 0 ? 0 : 0xffffffffu << (shift + bits);  // the bits already settled
#pragma unroll 4
    for (int j = lo + threadIdx.x; j < hi; j += S_THREADS) {
      const uint32_t key = order_key(w[j]);
      if ((key & above) == border) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1)], 1u);
    }
    cluster_sync_all();
    // every CTA adds up all of them: thread t the bins 4t .. 4t + 3 from the top
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int bin = S_BINS - 1 - (4 * (int)threadIdx.x + i);
      c[i] = 0;
#pragma unroll
      for (int r = 0; r < S_CTAS; ++r) c[i] += ld_cluster_u32(&hist[bin], r);
    }
    int total;
    uint32_t before = (uint32_t)block_scan((int)(c[0] + c[1] + c[2] + c[3]), warp_sums, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (before < take && take <= before + c[i]) {
        chosen[0] = (uint32_t)(S_BINS - 1 - (4 * (int)threadIdx.x + i));
        chosen[1] = take - before;
      }
      before += c[i];
    }
    cluster_sync_all();  // chosen is written; every CTA has read the histograms
    border |= chosen[0] << shift;
    take = chosen[1];
    __syncthreads();
  }

  // ---- how many each CTA keeps
  if (threadIdx.x < 2) counts[threadIdx.x] = 0;
  __syncthreads();
  uint32_t gt = 0, eq = 0;
#pragma unroll 4
  for (int j = lo + threadIdx.x; j < hi; j += S_THREADS) {
    const uint32_t key = order_key(w[j]);
    gt += key > border;
    eq += key == border;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&counts[0], gt);
    atomicAdd(&counts[1], eq);
  }
  cluster_sync_all();
  uint32_t at = 0, eq_before = 0;
  for (int r = 0; r < rank; ++r) {
    at += ld_cluster_u32(&counts[0], r);
    eq_before += ld_cluster_u32(&counts[1], r);
  }
  at += min(eq_before, take);
  cluster_sync_all();  // no CTA ends while its counts are read

  // ---- the kept positions in order, four a thread at a time
  for (int j0 = lo; j0 < hi; j0 += 4 * S_THREADS) {
    const int j = j0 + 4 * (int)threadIdx.x;
    float x[4];
    uint32_t key[4];
    int eqs = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = j + i < hi ? w[j + i] : 0.f;
      key[i] = order_key(x[i]);
      eqs += j + i < hi && key[i] == border;
    }
    int total;
    uint32_t e = eq_before + (uint32_t)block_scan(eqs, warp_sums, &total);
    eq_before += (uint32_t)total;
    bool keep[4];
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool same = j + i < hi && key[i] == border;
      keep[i] = j + i < hi && (key[i] > border || (same && e < take));
      e += same;
      n += keep[i];
    }
    uint32_t o = at + (uint32_t)block_scan(n, warp_sums, &total);
    at += (uint32_t)total;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (keep[i]) {
        kept[o] = j + i;
        wo[o] = x[i];
        ++o;
      }
  }
}

constexpr int M_THREADS = 256;
constexpr int M_PAGE = 256;  // most tokens of a page

__global__ void __launch_bounds__(M_THREADS) kv8_move_kernel(Kv8View v, EvictArgs a) {
  kv8_ready();
  __shared__ const int8_t* row_codes[M_PAGE];
  __shared__ float row_scale[M_PAGE];
  __shared__ float s_max[M_THREADS / 32];
  const int b = blockIdx.z, g = (int)(blockIdx.x % v.kv_heads), index = (int)(blockIdx.x / v.kv_heads);
  const bool is_v = blockIdx.y != 0;
  const int len = kv8_len(v, b);
  if (len <= a.budget) return;
  const int to = a.fresh[(size_t)b * a.fresh_w + index];
  if (to < 0 || to >= v.num_pages) {
    if (threadIdx.x == 0) kv8_flag(v);
    return;
  }
  const int* kept = a.kept + ((size_t)b * v.kv_heads + g) * a.budget + ((size_t)index << v.page_shift);
  const int rows = min(1 << v.page_shift, a.budget - (index << v.page_shift));
  int8_t* base = is_v ? v.V : v.K;
  float* scales = is_v ? v.v_scale : v.k_scale;
  const int vshift = 31 - __clz(v.dim / 16);
  const int mask = (1 << v.page_shift) - 1;
  for (int r = threadIdx.x; r < rows; r += M_THREADS) {
    const int j = kept[r];  // within 0 .. len - 1: written by the selection
    const int page = kv8_page(v, b, j >> v.page_shift);
    row_codes[r] = page < 0 ? nullptr : base + kv8_codes_at(v, page, g) + (size_t)(j & mask) * v.dim;
    row_scale[r] = page < 0 ? 0.f : scales[kv8_scale_at(v, page, g)];
  }
  __syncthreads();
  const int nvec = rows << vshift, cmask = (1 << vshift) - 1;
  auto load = [&](int i) {
    const int8_t* p = row_codes[i >> vshift];
    return p ? __ldg(reinterpret_cast<const uint4*>(p) + (i & cmask)) : make_uint4(0, 0, 0, 0);
  };
  float m = 0.f;
#pragma unroll 4
  for (int i = threadIdx.x; i < nvec; i += M_THREADS) {
    const uint4 w = load(i);
    // the largest |code| of the 16: rounding to float32 keeps order, so the
    // largest |value| is the value of the largest |code|
    uint32_t c = __vmaxu4(__vmaxu4(__vabs4(w.x), __vabs4(w.y)), __vmaxu4(__vabs4(w.z), __vabs4(w.w)));
    c = __vmaxu4(c, c >> 16);
    const uint32_t top = max(c & 255u, (c >> 8) & 255u);
    m = fmaxf(m, finite_abs((float)top * row_scale[i >> vshift]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < M_THREADS / 32; ++w) m = fmaxf(m, s_max[w]);
  const float s = kv8_scale_of(m), inv = __fdiv_rn(1.0f, s);
  if (threadIdx.x == 0) scales[kv8_scale_at(v, to, g)] = s;
  uint4* dst = reinterpret_cast<uint4*>(base + kv8_codes_at(v, to, g));
#pragma unroll 2
  for (int i = threadIdx.x; i < nvec; i += M_THREADS) {
    uint4 w = load(i);
    const float so = row_scale[i >> vshift];
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      int c[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) c[t] = kv8_code((float)kv8_byte(u[j], t) * so, s, inv);
      u[j] = kv8_pack4(c[0], c[1], c[2], c[3]);
    }
    dst[i] = w;
  }
}

}  // namespace

cudaError_t launch_kv8_evict(const Kv8View& v, const float* weights, long long weights_ld, int budget, int recent,
                             const int* fresh, int* table_out, int* lens_out, float* weights_out,
                             long long weights_out_ld, int* kept, cudaStream_t s) {
  const int page = 1 << v.page_shift, fresh_w = (int)(((long long)budget + page - 1) / page);
  const EvictArgs a{weights,   weights_ld, budget,      recent,         fresh_w, fresh,
                    table_out, lens_out,   weights_out, weights_out_ld, kept};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S_CTAS, (unsigned)v.kv_heads, (unsigned)v.num_seqs);
  cfg.blockDim = dim3(S_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {pdl_attr()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S_CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_select_kernel, v, a);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t mcfg = {};
  mcfg.gridDim = dim3((unsigned)fresh_w * v.kv_heads, 2, (unsigned)v.num_seqs);
  mcfg.blockDim = dim3(M_THREADS);
  mcfg.stream = s;
  mcfg.attrs = attr;
  mcfg.numAttrs = 1;
  return cudaLaunchKernelEx(&mcfg, kv8_move_kernel, v, a);
}

}  // namespace apr
