// Eviction from the 8-bit paged KV cache (include/apr_kv8.h): which positions
// a sequence keeps, and their move into fresh pages.
//
// Selection. One cluster of 1 to 8 CTAs per (sequence, KV head), each CTA a
// contiguous share of the positions, whose weights it reads once: mapped to
// unsigned keys that order as the numbers do they stay in shared memory (a
// share of more than 20480 is read again for each pass, from L2). The key of
// the last one kept is found by rounds of histograms over 11, 11 and 10 bits of
// it, in a cluster over 8 bits each time, whose counts every CTA adds up through
// distributed shared memory; a round whose border falls between two bins ends
// the search. The kept positions are then written in order: each CTA knows from
// its peers' counts how many come before its own, and of equal keys the lowest
// positions are taken. Every count is a whole number, so the result does not
// depend on the order of the atomics. Bound by instructions of the few SMs that
// it runs on (30700 keys by one: loads and first counts 7 us, rounds 4, the
// kept positions 7) and, below some thousand keys, by latency.
//
// Move. One CTA per (fresh page, KV head), K or V: the kept rows' codes are
// gathered into registers, their largest value gives the scale, and they are
// written under it, five instructions and a byte permute a value
// (kv8_requantise16). What a large page has more than the registers hold is
// gathered again, from L1. Bound by instructions and the way to the rows (kept
// position, page, scale, codes), which nine CTAs an SM cover for one another: K
// and V in one CTA, or several pages a CTA with the next one's rows gathered
// ahead, at 72 to 92 registers a thread, took longer.
//
// Measured (GB300): 10 sequences of 3500 to 33000 positions, 8 heads of 128, to
// 4100: selection 20 us (3.9 MB of weights: instructions, not bytes), move 45 us, 151
// MB (0.50 of the HBM rate).

#include "apr_internal.h"
#include "host_common.h"
#include "kv8.cuh"

namespace apr {
namespace {

constexpr int S_MOST = 8;        // CTAs of a cluster, the portable size
constexpr int S_THREADS = 1024;
constexpr int S_WARPS = S_THREADS / 32;
constexpr int S_BINS = 2048;
constexpr int S_KEYS = 20480;    // keys that a CTA holds

// Unsigned keys in the numbers' order: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float order_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, int rank) {
  uint32_t r;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(mapa_shared(smem_u32(p), (uint32_t)rank)) : "memory");
  return r;
}
// The barrier of a cluster of `ranks` CTAs.
__device__ __forceinline__ void cluster_sync_all(int ranks) {
  if (ranks == 1) {
    __syncthreads();
  } else {
    cluster_arrive();
    cluster_wait();
  }
}

// Sum of x over the threads before this one, and over all of them (*total).
// `sums` [S_WARPS] must not be in use by the scan before.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  uint32_t w = lane < S_WARPS ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp ? before : 0) + inc - x;
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

__global__ void __launch_bounds__(S_THREADS) kv8_select_kernel(const __grid_constant__ Kv8View v,
                                                               const __grid_constant__ EvictArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ uint32_t hist[S_BINS];
  __shared__ uint32_t chosen[2];  // the round's bin, and how many of it are kept
  __shared__ uint32_t counts[2];  // this CTA's keys above the border, and equal to it
  __shared__ uint32_t sums[2][S_WARPS];
  const int ranks = gridDim.x, rank = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int len = kv8_len(v, b);
  const size_t bg = (size_t)b * v.kv_heads + g;
  const float* w = a.weights + bg * a.weights_ld;
  float* wo = a.weights_out + bg * a.weights_out_ld;
  int* kept = a.kept + bg * a.budget;
  const int now = min(len, a.budget);
  const int all = ranks * S_THREADS, tid = rank * S_THREADS + threadIdx.x;
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
  const int share = (old + ranks - 1) / ranks;
  const int lo = min(rank * share, old), n = min(share, old - lo);
  w += lo;
  const bool held = share <= S_KEYS;
  for (int i = threadIdx.x; i < S_BINS; i += S_THREADS) hist[i] = 0;
  __syncthreads();
  // Bits of a key that a round settles: few bins where every CTA has to read all
  // the others', fewer rounds where it is alone (the whole call, us, 8 bits against
  // 11: 8 heads of 131000 positions 62 and 70, of 4 sequences of 60000 61 and 62,
  // 2 heads of 200000 46 and 52; alone, 4 heads of 4099, 15.4 and 14.3).
  const int width = ranks == 1 ? 11 : 8, top_shift = 32 - width;
  // the keys, and the first round's counts; the zeros, often the most, are
  // counted by the warp instead of one after the other in one bin
  constexpr uint32_t ZERO = 0x80000000u;
  constexpr int AT_ONCE = 8;
  for (int j0 = threadIdx.x; j0 < (n + 31) / 32 * 32; j0 += AT_ONCE * S_THREADS) {  // (whole warps)
    float x[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) x[i] = j0 + i * S_THREADS < n ? w[j0 + i * S_THREADS] : 1.f;
    int zeros = 0;
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int j = j0 + i * S_THREADS;
      const uint32_t key = order_key(x[i]);
      if (held && j < n) s_keys[j] = key;
      zeros += __popc(__ballot_sync(0xffffffffu, key == ZERO));
      if (j < n && key != ZERO) atomicAdd(&hist[key >> top_shift], 1u);
    }
    if ((threadIdx.x & 31) == 0 && zeros) atomicAdd(&hist[ZERO >> top_shift], (uint32_t)zeros);
  }
  auto key_at = [&](int j) { return held ? s_keys[j] : order_key(w[j]); };

  // ---- the key of the last position kept: border, of whose equals `take` are kept
  uint32_t border = 0, take = (uint32_t)need;
#pragma unroll 1
  for (int round = 0, bits, shift = 32; shift > 0; ++round) {
    bits = min(width, shift);
    shift -= bits;
    if (round > 0) {
      for (int i = threadIdx.x; i < 1 << bits; i += S_THREADS) hist[i] = 0;
      __syncthreads();
      const uint32_t above = 0xffffffffu << (shift + bits);  // the bits already settled
#pragma unroll 8
      for (int j = threadIdx.x; j < n; j += S_THREADS) {
        const uint32_t key = key_at(j);
        if ((key & above) == border) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1)], 1u);
      }
    }
    cluster_sync_all(ranks);
    // every CTA adds up all of them: thread t the bins PER t .. PER t + PER - 1 from the top
    constexpr int PER = S_BINS / S_THREADS;
    const int top = (1 << bits) - 1 - PER * (int)threadIdx.x;
    uint32_t c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = ranks == 1 && top - i >= 0 ? hist[top - i] : 0;
    if (ranks > 1 && top > 0) {
#pragma unroll
      for (int r = 0; r < S_MOST; ++r)
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (r < ranks) c[i] += ld_cluster_u32(&hist[top - i], r);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += c[i];
    uint32_t total;
    uint32_t before = block_scan(sum, sums[round & 1], &total);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (before < take && take <= before + c[i]) {
        chosen[0] = ((uint32_t)(top - i) << 1) | (take - before == c[i]);
        chosen[1] = take - before;
      }
      before += c[i];
    }
    cluster_sync_all(ranks);  // chosen is written; every CTA has read the histograms
    border |= (chosen[0] >> 1) << shift;
    take = chosen[1];
    if (chosen[0] & 1) {  // the whole bin is kept: the border lies just below it
      border -= 1;        // (not below 0: then every position would be kept)
      take = 0;
      break;
    }
  }

  // ---- how many of the CTAs before are kept
  uint32_t gt_before = 0, eq_before = 0;
  if (ranks > 1) {
    if (threadIdx.x < 2) counts[threadIdx.x] = 0;
    __syncthreads();
    uint32_t gt = 0, eq = 0;
#pragma unroll 8
    for (int j = threadIdx.x; j < n; j += S_THREADS) {
      const uint32_t key = key_at(j);
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
    cluster_sync_all(ranks);
    for (int r = 0; r < rank; ++r) {
      gt_before += ld_cluster_u32(&counts[0], r);
      eq_before += ld_cluster_u32(&counts[1], r);
    }
    cluster_sync_all(ranks);  // no CTA ends while its counts are read
  }
  __syncthreads();

  // ---- the kept positions in order, some neighbours a thread at a time; the
  // scan counts those above the border in its low half, those equal in its high
  constexpr int RUN = 8;
  int half = 0;
  for (int j0 = 0; j0 < n; j0 += RUN * S_THREADS, half ^= 1) {
    const int j = j0 + RUN * (int)threadIdx.x;
    uint32_t key[RUN], mine = 0;
    if (held && j < n) {  // (the keys' array ends on a whole run)
#pragma unroll
      for (int i = 0; i < RUN; i += 4) *reinterpret_cast<uint4*>(key + i) = *reinterpret_cast<const uint4*>(s_keys + j + i);
    }
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      if (!held) key[i] = j + i < n ? order_key(w[j + i]) : 0u;
      mine += j + i < n ? (key[i] > border ? 1u : (key[i] == border ? 1u << 16 : 0u)) : 0u;
    }
    uint32_t total;
    const uint32_t before = block_scan(mine, sums[half], &total);
    uint32_t gt = gt_before + (before & 0xffffu), eq = eq_before + (before >> 16);
    gt_before += total & 0xffffu;
    eq_before += total >> 16;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      if (j + i >= n) break;
      const bool same = key[i] == border;
      if (key[i] > border || (same && eq < take)) {
        const uint32_t o = gt + min(eq, take);
        kept[o] = lo + j + i;
        wo[o] = order_value(key[i]);
      }
      gt += key[i] > border;
      eq += same;
    }
  }
}

constexpr int M_THREADS = 128;
constexpr int M_PAGE = 256;  // most tokens of a page
constexpr int M_HELD = 4;    // vectors of 16 codes that a thread holds

// The largest |code| of a vector times its scale: rounding to float32 keeps
// order, so that is the largest |value|. Two codes at a time, sign-extended to
// 16 bits by one byte permute.
__device__ __forceinline__ float amax_of_codes(const uint4& in, float scale) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  uint32_t top = 0, low = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a, b;  // (8 + i in a selector repeats byte i's sign)
    asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(w[i]));
    asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(b) : "r"(w[i]));
    top = __vimax3_s16x2(top, a, b);
    low = __vimin3_s16x2(low, a, b);
  }
  const int hi = max((int)(int16_t)top, (int)top >> 16), lo = min((int)(int16_t)low, (int)low >> 16);
  return finite_abs((float)max(hi, -lo) * scale);
}

template <int D>
__global__ void __launch_bounds__(M_THREADS) kv8_move_kernel(const __grid_constant__ Kv8View v,
                                                             const __grid_constant__ EvictArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ long long row_at[M_PAGE];  // offset of a row's codes; -1: none
  __shared__ float row_scale[M_PAGE];
  __shared__ float s_max[M_THREADS / 32];
  const bool is_v = blockIdx.x & 1;  // K and V of a page are neighbours: they look up the same rows
  const int b = blockIdx.y, g = (int)((blockIdx.x >> 1) % v.kv_heads), index = (int)((blockIdx.x >> 1) / v.kv_heads);
  const int len = kv8_len(v, b);
  const int to = len > a.budget ? a.fresh[(size_t)b * a.fresh_w + index] : -1;
  if (len > a.budget && (to < 0 || to >= v.num_pages) && threadIdx.x == 0) kv8_flag(v);
  if (to < 0 || to >= v.num_pages) return;
  const int* kept = a.kept + ((size_t)b * v.kv_heads + g) * a.budget + ((size_t)index << v.page_shift);
  const int rows = min(1 << v.page_shift, a.budget - (index << v.page_shift));
  int8_t* codes = is_v ? v.V : v.K;
  float* scales = is_v ? v.v_scale : v.k_scale;
  constexpr int ROW = D / 16;  // vectors of a row
  for (int r = threadIdx.x; r < rows; r += M_THREADS) {
    const int j = kept[r];  // within 0 .. len - 1: written by the selection
    const int page = kv8_page(v, b, j >> v.page_shift);
    row_at[r] = page < 0 ? -1 : (long long)(kv8_codes_at(v, page, g) + (size_t)(j & ((1 << v.page_shift) - 1)) * D);
    row_scale[r] = page < 0 ? 0.f : scales[kv8_scale_at(v, page, g)];
  }
  __syncthreads();
  const int nvec = rows * ROW, col = (int)threadIdx.x % ROW * 16;
  auto load = [&](int i) {
    const long long at = row_at[i / ROW];
    return at < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(codes + at + col);
  };
  uint4 keep[M_HELD];
#pragma unroll
  for (int j = 0; j < M_HELD; ++j) {
    const int i = threadIdx.x + j * M_THREADS;
    keep[j] = i < nvec ? load(i) : make_uint4(0, 0, 0, 0);
  }
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < M_HELD; ++j) {
    const int i = threadIdx.x + j * M_THREADS;
    if (i < nvec) m = fmaxf(m, amax_of_codes(keep[j], row_scale[i / ROW]));
  }
  for (int i = threadIdx.x + M_HELD * M_THREADS; i < nvec; i += M_THREADS)
    m = fmaxf(m, amax_of_codes(load(i), row_scale[i / ROW]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < M_THREADS / 32; ++w) m = fmaxf(m, s_max[w]);
  const Kv8Scale s = kv8_rounding_to(kv8_scale_of(m));
  if (threadIdx.x == 0) scales[kv8_scale_at(v, to, g)] = s.s;
  uint4* dst = reinterpret_cast<uint4*>(codes + kv8_codes_at(v, to, g));
#pragma unroll
  for (int j = 0; j < M_HELD; ++j) {
    const int i = threadIdx.x + j * M_THREADS;
    if (i < nvec) dst[i] = kv8_requantise16(keep[j], row_scale[i / ROW], s);
  }
#pragma unroll 1
  for (int i = threadIdx.x + M_HELD * M_THREADS; i < nvec; i += M_THREADS)
    dst[i] = kv8_requantise16(load(i), row_scale[i / ROW], s);
}

}  // namespace

cudaError_t launch_kv8_evict(const Kv8View& v, const float* weights, long long weights_ld, int budget, int recent,
                             const int* fresh, int* table_out, int* lens_out, float* weights_out,
                             long long weights_out_ld, int* kept, cudaStream_t s) {
  const int page = 1 << v.page_shift, fresh_w = (int)(((long long)budget + page - 1) / page);
  const EvictArgs a{weights,   weights_ld, budget,      recent,         fresh_w, fresh,
                    table_out, lens_out,   weights_out, weights_out_ld, kept};
  // As few CTAs of a cluster as hold the keys of the longest sequence. One SM
  // takes about 0.6 us per 1000 keys for its passes, a cluster of two or more some
  // 6 us for its barriers (10 sequences of up to 33000, 8 heads, the eviction and
  // read-back: 105 us with two CTAs each, 109 with one, 118 with four).
  int ranks = 1;
  while (ranks < S_MOST && (v.max_len + ranks - 1) / ranks > S_KEYS) ranks *= 2;
  const int share = (v.max_len + ranks - 1) / ranks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ranks, (unsigned)v.kv_heads, (unsigned)v.num_seqs);
  cfg.blockDim = dim3(S_THREADS);
  cfg.dynamicSmemBytes = (size_t)(share < S_KEYS ? (share + 7) / 8 * 8 : S_KEYS) * sizeof(uint32_t);  // whole runs
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {pdl_attr()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  static bool ready[64] = {};  // the attribute is set once for each device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64 || !ready[dev])) {
    e = cudaFuncSetAttribute(kv8_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S_KEYS * (int)sizeof(uint32_t));
    if (e == cudaSuccess && dev >= 0 && dev < 64) ready[dev] = true;
  }
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kv8_select_kernel, v, a);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t mcfg = {};
  mcfg.gridDim = dim3(2u * fresh_w * v.kv_heads, (unsigned)v.num_seqs);
  mcfg.blockDim = dim3(M_THREADS);
  mcfg.stream = s;
  mcfg.attrs = attr;
  mcfg.numAttrs = 1;
  if (v.dim == 64) return cudaLaunchKernelEx(&mcfg, kv8_move_kernel<64>, v, a);
  if (v.dim == 128) return cudaLaunchKernelEx(&mcfg, kv8_move_kernel<128>, v, a);
  return cudaLaunchKernelEx(&mcfg, kv8_move_kernel<256>, v, a);
}

}  // namespace apr
