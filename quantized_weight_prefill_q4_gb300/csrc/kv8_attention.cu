// Attention of a sequence's last rows over its 8-bit paged KV cache
// (include/apr_kv8.h):
//   p_j = softmax_j(scale q . (c_j s)),  out = sum_j p_j (c'_j s'),  w_j = sum of p_j
//
// Bound. One byte of K or V enters 2 operations for each (row, head) pair that
// reads it, 8 pairs in a decode step of usual grouping: 16 operations a byte,
// far below the tensor cores' ratio, far above the CUDA cores' (float32 FMAs at
// the HBM rate: 6.7 TB/s x 16 = 107 TFLOP/s). So the products go to the tensor
// cores as m16n8k16 steps with 8 pairs as the M side, and what has to be kept
// below the HBM time is the rest: two byte permutes, an exclusive or and two
// subtractions for each four codes turned into fp16, which holds them exactly.
//
// Precision for free. The M side has 16 rows and 8 pairs, so each pair's
// float32 query (scaled by a power of two) goes in as two fp16 rows, q = hi +
// lo to 22 bits, and each softmax weight likewise: the two rows' results are
// added in float32. The sums over positions restart every TILE positions and
// are added up in float32 with the page's V scale, so the tensor cores never
// accumulate over a long sequence. A weight is kept times 2^10 against a
// reference that trails the running maximum by at most 4 (base 2), so weights
// down to 2^-34 of the largest keep a bit.
//
// Work. The pairs of a sequence that read the same KV head are taken PAIRS =
// 8 MT at a time; one such group of pairs over all the sequence's positions is
// a segment, and its positions go in units of UNIT. The units of all segments
// are numbered through, and each CTA takes an equal, contiguous share of them,
// so that sequences of any lengths in one batch keep every SM equally busy. A
// segment within one CTA's share is finished there; otherwise each CTA that has
// a piece of it writes the piece's unnormalised sums with their reference
// maximum and total, and a second kernel combines the pieces in order, a CTA for
// each pair. (Having the last CTA of a segment combine them instead took 3 to 9
// us more at the end of the measured cases: a fence behind every piece, and one
// CTA's loads instead of all SMs'.) Where the weights are wanted, more CTAs of the
// second kernel turn the scores that the first one kept into them.
//
// A CTA. Its warps take the piece's tiles of TILE positions in turn, each for
// all the segment's pairs. A warp streams its tiles through a ring of its own in
// shared memory by asynchronous 16-byte copies (a tile's K, its V, the next
// tile's K, ...), so that warps do not wait for one another before the piece's
// end, and the next piece's first chunks are on their way by then. A row's
// 16-byte chunks are stored exclusive-or'ed with bits of the row so that both
// products' reads are free of bank conflicts: for K a quarter warp reads 4
// chunks of 2 neighbouring rows, for V 2 chunks of every other row of 8.
// Lane (r, c) = (lane / 4, lane % 4) reads K's row 8 t + r, dims 16 c .. + 15 of
// each 64: word w holds its 4 dims of k-step w, an order of the dims that the
// query's fragments share. For V it reads dims 16 r .. + 15 of each 128 of the
// four rows 16 j + 2 c + {0, 1, 8, 9} that its weights belong to, and word w's
// byte t of them is its part of the product's columns 4 w + t.
//
// The softmax works in base 2.
//
// Measured (GB300, back to back in a graph): 48 sequences of 130 to 9000 tokens,
// 32 heads over 8 of 128: 45 us, 207 MB (0.69 of the HBM rate); 3 of 100000 to
// 131000, 16 over 4 of 256: 119 us (0.88), one of 700: 10.7 us; with weights 16 of
// 2000 to 12000, 32 over 4 of 128: 31 us, and 9 rows of each of 4 of 5000 to 8200,
// 16 over 8 of 64: 28 us. Of the 45 us the tiles stream at 6.3 TB/s for 33;
// the rest is the way to the first codes (length, table, codes: 3 us), CTAs of
// equal shares that end up to 5 us apart, and the combination (3 us). The 9 rows
// (18 pairs) are bound by the warps' instructions, 330 a tile and 8 pairs.

#include "apr_internal.h"
#include "host_common.h"
#include "kv8.cuh"

namespace apr {
namespace {

constexpr int UNIT = 64;      // positions of a unit of work
constexpr int MOST_UNITS = 1 << 30;  // of a call, as its arguments are checked for
// Where max_len * dim is at most this, segments are not divided among CTAs, which
// saves the second launch (about 4 us of the host's time where the calls follow one
// another): one sequence, 8 heads of 128, 200 / 512 / 700 positions 6.8 / 9.0 /
// 11.3 us on the device, divided 8.0 / 8.4 / 8.5; 64 sequences 16.2 / 24.1 / 30.4
// and 18.5 / 24.9 / 28.7. At 256 dims the sides meet at half the length.
constexpr int WHOLE_SIZE = 512 * 128;
// With weights there is a second launch either way, and what stays undivided saves
// only its combination. Where a KV head's pairs are one segment, dividing pays from
// less on: 1 / 8 / 64 sequences of 500 positions, one row, 8 heads of 128, 12.3 / 15.0
// / 29.7 us whole, 9.7 / 12.9 / 26.9 divided; of 1000, 64 dims, 13.3 / 16.2 / 29.9 and
// 8.9 / 12.2 / 27.7; of 200, 128 dims, 10.1 / 13.1 / 20.1 and 9.4 / 12.4 / 20.7; of 100,
// 9.4 / 10.1 / 17.1 and 9.6 / 11.9 / 17.9. With more segments the pieces cost more
// (32 rows, 500 positions of 128: 34.7 / 54.5 whole, 42.3 / 68.2 divided), at 256
// dims too (64 of 256, 17.7 and 22.5).
constexpr int WHOLE_SIZE_WEIGHTED = 192 * 128;
constexpr int MIN_SHARE = 2;  // units of a CTA's share, where there are not enough for every CTA
// Units that a segment counts for besides its positions: what its start (the
// way from the length over the page table to the codes, the query rows) and
// its end (the warps' sums) take, in units of 128 D bytes. (48 ragged
// sequences: 49 us with half as much, 44 with this or twice as much.)
__host__ __device__ constexpr int overhead_units(int dim) { return 512 / dim; }
constexpr int TILE = 32;      // positions of a tile, within one page
constexpr float HEADROOM = 10.f;  // weights are kept times 2^10
constexpr float MOVE_ABOVE = 4.f;  // the reference moves when the maximum is more than this above it
// V's scales enter times 2^-24, which the end takes back: of unnormalised weights,
// 2^10 and more each, the sum over 1000 values of 2^108 would pass float32's
// range (exact for scales from 2^-102 on, below which a value's last bits go).
constexpr float V_DOWN = 0x1p-24f, V_UP = 0x1p24f;

struct AttnArgs {
  Kv8View v;
  const void* q;
  void* out;
  long long ldq, ldo;
  int type, heads, group;
  int pairs;         // (row, head) pairs of a segment
  float scale_log2;  // softmax scale times log2(e)
  int ctas;          // of the grid; no more than there are units share them
  int whole;         // segments are not divided (WHOLE_SIZE)
  int* prefix;       // [num_seqs + 1] first unit of each sequence, all units (written by CTA 0)
  float2* part_ml;   // [2 ctas][pairs] reference maximum and total of a piece
  float* part_o;     // [2 ctas][pairs][dim]
  // For the weights, or nullptr. A sequence's (row, head) pairs are in the order
  // of the KV heads they read, pair_at() says where.
  float2* final_ml;  // [rows * heads] maximum and 1 / total
  float* scores;     // [rows * heads][scores_ld] scores in base 2
  int scores_ld;     // max_len rounded up to whole tiles
  float* weights;
  long long weights_ld;
  int accumulate;
};

// Units of one segment of a sequence (the overhead's first), and its segments.
__device__ __forceinline__ int segment_units(const AttnArgs& a, int len) {
  return overhead_units(a.v.dim) + max(1, (len + UNIT - 1) / UNIT);
}
__device__ __forceinline__ int segment_count(const AttnArgs& a, int n) {
  return (n * a.group + a.pairs - 1) / a.pairs * a.v.kv_heads;
}
__device__ __forceinline__ int sequence_units(const AttnArgs& a, int b) {
  const int n = kv8_rows(a.v, b).n;
  return n == 0 ? 0 : segment_count(a, n) * segment_units(a, kv8_len(a.v, b));
}

// CTAs that share `total` units, MIN_SHARE at least each (fewer share nothing).
__device__ __forceinline__ int sharing_ctas(const AttnArgs& a, int total) {
  return min(a.ctas, (total + MIN_SHARE - 1) / MIN_SHARE);
}

// Of `ctas` CTAs that share `total` units, CTA c has the units first_unit(c) .. first_unit(c + 1) - 1 of `total`; the
// CTA that has unit u.
__device__ __forceinline__ int first_unit(int c, int ctas, int total) {
  return (int)((long long)c * total / ctas);
}
__device__ __forceinline__ int cta_of(int u, int ctas, int total) {
  return (int)((((long long)u + 1) * ctas - 1) / total);
}

// ---------------------------------------------------------------- the tiles
// Where 16-byte chunk x of a tile (row x / (D / 16)) lies in its slot.
template <int D>
__device__ __forceinline__ int swizzled(int x) {
  const int row = x / (D / 16);
  const int bits = D >= 128 ? (((row ^ (row >> 1)) & 1) << 2) | (((row >> 2) & 1) << 1)
                            : (((row >> 1) & 1) << 2) | (((row >> 2) & 1) << 1);
  return x ^ bits;
}

__device__ __forceinline__ void copy_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D += A . B, m16n8k16, fp16 in, float32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// 4 consecutive elements of a row.
__device__ __forceinline__ float4 load4_any(const void* p, int type, size_t i) {
  if (type == APR_T_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  if (type == APR_T_F16) {
    const float2 a = half2_values(w.x), b = half2_values(w.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

__device__ __forceinline__ void store4_any(void* p, int type, size_t i, const float4& x) {
  if (type == APR_T_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = x;
  } else if (type == APR_T_F16) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(half2_bits(x.x, x.y), half2_bits(x.z, x.w));
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// What a piece's sums and total are to be multiplied by under the reference m.
__device__ __forceinline__ float piece_factor(float2 ml, float m) {
  return ml.y > 0.f ? exp2f(ml.x - m) : (ml.y != ml.y ? 1.f : 0.f);
}
// Where the weights' arrays have pair 0 of a sequence's rows and KV head.
__device__ __forceinline__ size_t pair_at(const AttnArgs& a, int r0, int n, int g) {
  return (size_t)r0 * a.heads + (size_t)g * n * a.group;
}

// Four dims from d of a (row, head)'s output, from its unnormalised sums and total.
__device__ __forceinline__ void finish4(const AttnArgs& a, int r0, int n, int g, int pair, int dim, int d,
                                        const float4& o, float m, float total) {
  const float inv = total > 0.f || total != total ? 1.f / total : 0.f;  // no position seen: zeros
  const size_t row = r0 + pair / a.group, head = g * a.group + pair % a.group;
  const float up = inv * V_UP;
  store4_any(a.out, a.type, row * a.ldo + head * dim + d, make_float4(o.x * up, o.y * up, o.z * up, o.w * up));
  if (a.final_ml && d == 0) a.final_ml[pair_at(a, r0, n, g) + pair] = make_float2(m, inv);
}

// A warp's M tiles, MT: 1, or 2 where that leaves less to do for the longest
// row group of a sequence: the codes are turned into fp16 once for both tiles,
// so that a segment of two costs about 1.5 of one (16 pairs over 4 x 60000
// positions of 128 dims: 112 us, 140 as two segments; 18 pairs over 4 x 8000 of
// 64: 32 us, 29 as three). Only up to 128 dims, where the registers hold the sums
// of 16 pairs. Where max_rows is left out the mean of the rows decides, not all of
// the call's (48 ragged sequences of one row: 46 us, 65 with two tiles). (The warps
// of a CTA sharing tiles between them, 8 pairs each, took longer than more segments
// for any number of pairs: 152 us for the 16.)
__host__ __device__ constexpr int m_tiles(int dim, long long pairs) {
  return dim <= 128 && (pairs + 15) / 16 * 3 < (pairs + 7) / 8 * 2 ? 2 : 1;
}

// CTAs of 4 warps on an SM, as registers (168 a thread, 255; 16 to 68 bytes of them
// spilled, but for 64 dims and one M tile) and shared memory allow. (At 128 dims 16 warps of 128 registers took 96 us for 4 sequences of
// 60000 where 12 take 83.)
constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
__host__ __device__ constexpr int ctas_per_sm(int dim, int mt) { return dim == 64 || (dim == 128 && mt == 1) ? 3 : 2; }

template <int D, int MT>
struct Shape {
  static constexpr int PAIRS = 8 * MT;
  static constexpr int SLOT = TILE * D;     // bytes of a tile's K or V
  static constexpr int SLOTS = 3;           // of a warp's ring
  static constexpr int STEPS = D / 16;      // k-steps of a score
  static constexpr int OFF_Q = WARPS * SLOTS * SLOT;
  // A warp's sums of an M tile, 8 rows, are as large as a slot: those of the
  // first lie in the last slot of its own ring, which the next piece's first
  // chunks do not use.
  static constexpr int OFF_M = OFF_Q + MT * STEPS * 512;
  static constexpr int BYTES = OFF_M + (MT - 1) * WARPS * SLOT;
  static_assert(8 * D * 4 == SLOT, "a warp's sums fill a slot");
};

template <int D, int MT>
__global__ void __launch_bounds__(THREADS, ctas_per_sm(D, MT))
    kv8_attention_kernel(const __grid_constant__ AttnArgs a) {
  using S = Shape<D, MT>;
  grid_dependency_wait();
  // (The next kernel is let in late: launched at once, its CTAs took the places of
  // this grid's as they freed up, and those of the next call's grid found some SMs
  // full; 48 ragged sequences 64 us, against 50 without.)
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long s_scan[WARPS];
  __shared__ int s_find[2];
  __shared__ float s_factor[S::PAIRS];          // score of a pair = factor * (K scale) * sum of products
  __shared__ float2 s_ml[WARPS][S::PAIRS];
  const Kv8View& v = a.v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * S::SLOTS * S::SLOT;
  const uint32_t ring_u32 = smem_u32(ring);
  const uint4* sq = reinterpret_cast<const uint4*>(smem + S::OFF_Q) + lane;

  // ---- the units of the sequences, and where this CTA's share begins: a
  // thread counts the units of `run` neighbouring sequences
  const int run = (v.num_seqs + THREADS - 1) / THREADS;
  const int my_b0 = min((int)threadIdx.x * run, v.num_seqs), my_b1 = min(my_b0 + run, v.num_seqs);
  long long my_units = 0;
  for (int b = my_b0; b < my_b1; ++b) my_units += sequence_units(a, b);
  long long inc = my_units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  long long my_u0 = inc - my_units, all_units = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) my_u0 += s_scan[w];
    all_units += s_scan[w];
  }
  // more than the host allows for: row ranges that overlap
  const int total = all_units <= MOST_UNITS ? (int)all_units : 0;
  if (all_units > MOST_UNITS && threadIdx.x == 0) kv8_flag(v);
  if (blockIdx.x == 0) {
    int at = (int)my_u0;
    for (int b = my_b0; b < my_b1; ++b) {
      a.prefix[b] = at;
      at += sequence_units(a, b);
    }
    if (threadIdx.x == 0) a.prefix[v.num_seqs] = total;
  }
  const int ctas = sharing_ctas(a, total);
  if ((int)blockIdx.x >= ctas) return;
  int u = first_unit(blockIdx.x, ctas, total);
  const int u_begin = u, u_end = first_unit(blockIdx.x + 1, ctas, total);
  if (my_u0 <= u && u < my_u0 + my_units) {
    int b = my_b0, at = (int)my_u0;
    for (int n; b + 1 < my_b1 && at + (n = sequence_units(a, b)) <= u; ++b) at += n;
    s_find[0] = b;
    s_find[1] = at;
  }
  __syncthreads();
  int b = s_find[0], seq_u0 = s_find[1];

  // ---- the piece of work at hand
  int len, g, p0, np, first, seg_end, ue, k0, mine;
  Kv8Span span;
  uint32_t at_next = 0;           // lane i: the place in the cache, in tiles, of the warp's tile 32 n + i
  float ks_all = 0.f, vs_all = 0.f;  // and its scales
  constexpr int QP = S::PAIRS / WARPS, QV = (D + 127) / 128;
  float4 x[QP][QV];               // the pairs' query rows, on their way

  const int in_page = (1 << v.page_shift) / TILE - 1;
  // (page ids out of range read page 0, and are flagged)
  auto tile_of = [&](int i, size_t* scale_at) {
    const int k = k0 + (warp + min(i, mine - 1) * WARPS) * TILE;
    const int page = max(kv8_page(v, b, k >> v.page_shift), 0);
    *scale_at = kv8_scale_at(v, page, g);
    return (uint32_t)(*scale_at << (v.page_shift - 5)) + (uint32_t)((k / TILE) & in_page);
  };
  // sends chunk n of the warp's (tile n / 2; its K, then its V) into the ring
  auto send = [&](int n) {
    if (n < 2 * mine) {
      const int i = n >> 1;
      if ((n & 63) == 0 && n) {
        size_t scale_at;
        at_next = tile_of(i + lane, &scale_at);
      }
      const uint32_t at = __shfl_sync(0xffffffffu, at_next, i & 31);
      const int8_t* src = (n & 1 ? v.V : v.K) + (size_t)at * S::SLOT;
      const uint32_t dst = ring_u32 + (n % S::SLOTS) * S::SLOT;
#pragma unroll
      for (int j = 0; j < S::SLOT / 512; ++j) {
        const int y = j * 32 + lane;
        copy_async_16(dst + swizzled<D>(y) * 16, src + y * 16);
      }
    }
    copy_commit();
  };
  // the next piece of this CTA's share, if there is one: its first tiles and its query rows under way
  auto begin = [&]() -> bool {
    for (;;) {
      if (u >= u_end || b >= v.num_seqs) return false;
      len = kv8_len(v, b);
      span = kv8_rows(v, b);
      const int su = segment_units(a, len), nseg = span.n ? segment_count(a, span.n) : 0;
      if (u >= seq_u0 + nseg * su) {  // the next sequence that has rows
        seq_u0 += nseg * su;
        ++b;
        continue;
      }
      const int seg = (u - seq_u0) / su, seg_u0 = seq_u0 + seg * su;
      g = seg % v.kv_heads;
      p0 = seg / v.kv_heads * S::PAIRS;
      np = min(S::PAIRS, span.n * a.group - p0);
      first = seg_u0 + overhead_units(D);  // the segment's first unit of positions
      seg_end = seg_u0 + su;
      if (a.whole && u > seg_u0) {  // of whole segments, those that begin in the share
        u = seg_end;
        continue;
      }
      ue = a.whole ? seg_end : min(u_end, seg_end);
      if (ue > first) break;
      u = ue;  // nothing but overhead: the next CTA begins the segment
    }
    k0 = max(u - first, 0) * UNIT;
    const int k1 = min(len, (ue - first) * UNIT);
    // this warp's tiles: every WARPS-th of the piece's
    const int tiles = k1 > k0 ? (k1 - k0 + TILE - 1) / TILE : 0;
    mine = tiles > warp ? (tiles - warp + WARPS - 1) / WARPS : 0;
    if (mine > 0) {
      size_t scale_at;
      at_next = tile_of(lane, &scale_at);
      ks_all = v.k_scale[scale_at];
      vs_all = v.v_scale[scale_at];
    }
#pragma unroll
    for (int i = 0; i < QP; ++i) {
      const int p = warp + i * WARPS, pair = p0 + p;
      const size_t row = span.r0 + pair / a.group, head = g * a.group + pair % a.group;
#pragma unroll
      for (int j = 0; j < QV; ++j) {
        const int d = 128 * j + 4 * lane;
        x[i][j] = p < np && d < D ? load4_any(a.q, a.type, row * a.ldq + head * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int n = 0; n < S::SLOTS - 1; ++n) send(n);
    return true;
  };

  bool more = begin();
  while (more) {
    // ---- the rows as fragments: row r of an M tile its fp16 hi, row r + 8 its lo
#pragma unroll
    for (int i = 0; i < QP; ++i) {
      const int p = warp + i * WARPS;
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < QV; ++j)
        top = fmaxf(top, fmaxf(fmaxf(fabsf(x[i][j].x), fabsf(x[i][j].y)), fmaxf(fabsf(x[i][j].z), fabsf(x[i][j].w))));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // the power of two that brings the largest magnitude into [1, 2) (kept
      // to 2^+-120: beyond, the row enters scaled less, its products still in range)
      const int e = top <= FLT_MAX ? min(max((int)(__float_as_uint(top) >> 23) - 127, -120), 120) : 0;
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      if (lane == 0) s_factor[p] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int j = 0; j < QV; ++j) {
        const int d = 128 * j + 4 * lane;
        if (d < D) {
          const float4 y = make_float4(x[i][j].x * down, x[i][j].y * down, x[i][j].z * down, x[i][j].w * down);
          const uint32_t h0 = half2_bits(y.x, y.y), h1 = half2_bits(y.z, y.w);
          const float2 f0 = half2_values(h0), f1 = half2_values(h1);
          const int step = d / 64 * 4 + d % 16 / 4, col = d % 64 / 16;
          reinterpret_cast<uint4*>(smem + S::OFF_Q)[((p / 8) * S::STEPS + step) * 32 + (p % 8) * 4 + col] =
              make_uint4(h0, half2_bits(y.x - f0.x, y.y - f0.y), h1, half2_bits(y.z - f1.x, y.w - f1.y));
        }
      }
    }
    __syncthreads();

    // this lane's pairs: row r of each M tile
    int limit[MT];        // positions that the pair sees
    float factor[MT];
    float* score_row[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int pair = p0 + 8 * t + r;
      const bool live = 8 * t + r < np;
      limit[t] = live ? min(len, len - span.n + pair / a.group + 1) : 0;
      factor[t] = s_factor[8 * t + r];
      score_row[t] = nullptr;
      if (a.scores && live)
        score_row[t] = a.scores + (pair_at(a, span.r0, span.n, g) + pair) * a.scores_ld + 2 * c;
    }
    const int least = len - span.n + p0 / a.group + 1;  // the fewest of these pairs'

    float ref[MT], l[MT];
    float2 sum[MT][D / 8];  // [column 4 w + t of each 128 dims]: dims 32 c + (4 w + t) and + 16 (D = 64: 16 c and + 8)
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      ref[t] = -INFINITY;
      l[t] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) sum[t][i] = make_float2(0.f, 0.f);
    }

#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      if ((i & 31) == 0 && i) {
        size_t scale_at;
        tile_of(i + lane, &scale_at);
        ks_all = v.k_scale[scale_at];
        vs_all = v.v_scale[scale_at];
      }
      const float ks = __shfl_sync(0xffffffffu, ks_all, i & 31), vs = __shfl_sync(0xffffffffu, vs_all, i & 31) * V_DOWN;
      const int k = k0 + (warp + i * WARPS) * TILE;

      // ---- scores of the tile's 32 positions: 4 columns of 8
      copy_wait<S::SLOTS - 2>();
      __syncwarp();
      send(2 * i + S::SLOTS - 1);
      const uint8_t* kt = ring + (2 * i) % S::SLOTS * S::SLOT;
      float s[MT][4][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t) s[m][t][0] = s[m][t][1] = s[m][t][2] = s[m][t][3] = 0.f;
#pragma unroll
      for (int d64 = 0; d64 < D / 64; ++d64) {
        uint4 kw[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          kw[t] = *reinterpret_cast<const uint4*>(kt + swizzled<D>((8 * t + r) * (D / 16) + 4 * d64 + c) * 16);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint4 qa[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) qa[m] = sq[(m * S::STEPS + 4 * d64 + w) * 32];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t x = (w == 0 ? kw[t].x : w == 1 ? kw[t].y : w == 2 ? kw[t].z : kw[t].w) ^ 0x80808080u;
            const uint32_t b0 = half2_of_codes(x, 0x4140), b1 = half2_of_codes(x, 0x4342);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma16816(s[m][t], qa[m], b0, b1);
          }
        }
      }

      // ---- the softmax weights
      uint4 pa[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float kf = ks * factor[m];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float2 both = __fmul2_rn(__fadd2_rn(make_float2(s[m][t][0], s[m][t][1]), make_float2(s[m][t][2], s[m][t][3])),
                                         make_float2(kf, kf));
          s[m][t][0] = both.x;
          s[m][t][1] = both.y;
        }
        if (k + TILE > least) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int j = k + 8 * t + 2 * c;
            if (j >= limit[m]) s[m][t][0] = -INFINITY;
            if (j + 1 >= limit[m]) s[m][t][1] = -INFINITY;
          }
        }
        if (score_row[m]) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
            *reinterpret_cast<float2*>(score_row[m] + k + 8 * t) = make_float2(s[m][t][0], s[m][t][1]);
        }
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t) top = fmaxf(top, fmaxf(s[m][t][0], s[m][t][1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (__any_sync(0xffffffffu, top > ref[m] + MOVE_ABOVE)) {
          const float now = fmaxf(ref[m], top);
          const float f = ref[m] == -INFINITY ? 0.f : exp2_fast(ref[m] - now);
          l[m] *= f;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) sum[m][j] = __fmul2_rn(sum[m][j], make_float2(f, f));
          ref[m] = now;
        }
        const float shift = ref[m] == -INFINITY ? 0.f : ref[m] - HEADROOM;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x = exp2_fast(s[m][2 * j + h][0] - shift), y = exp2_fast(s[m][2 * j + h][1] - shift);
            l[m] += x + y;
            hi[h] = half2_bits(x, y);
            const float2 f = half2_values(hi[h]);
            lo[h] = half2_bits(x - f.x, y - f.y);
          }
          pa[m][j] = make_uint4(hi[0], lo[0], hi[1], lo[1]);
        }
      }

      // ---- their product with the tile's V
      copy_wait<S::SLOTS - 2>();
      __syncwarp();
      send(2 * i + S::SLOTS);
      const uint8_t* vt = ring + (2 * i + 1) % S::SLOTS * S::SLOT;
      constexpr int COLS = D >= 128 ? 16 : 8;  // columns a lane's bytes of a row give
#pragma unroll
      for (int dc = 0; dc < (D + 127) / 128; ++dc) {
        uint32_t vw[2][4][COLS / 4];  // [k-step][row 2 c + {0, 1, 8, 9}][words]
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int row = 16 * j + 2 * c + (h & 1) + 8 * (h >> 1);
            if (D >= 128) {
              *reinterpret_cast<uint4*>(vw[j][h]) =
                  *reinterpret_cast<const uint4*>(vt + swizzled<D>(row * (D / 16) + 8 * dc + r) * 16);
            } else {
              *reinterpret_cast<uint2*>(vw[j][h]) =
                  *reinterpret_cast<const uint2*>(vt + swizzled<D>(row * (D / 16) + r / 2) * 16 + (r & 1) * 8);
            }
          }
#pragma unroll
        for (int w = 0; w < COLS / 4; ++w) {
          float o[MT][4][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < 4; ++t) o[m][t][0] = o[m][t][1] = o[m][t][2] = o[m][t][3] = 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t x[2][2];  // [rows 2 c, 2 c + 1 or + 8][columns 0, 1 or 2, 3]: the two rows' bytes side by side
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              x[h][0] = __byte_perm(vw[j][2 * h][w], vw[j][2 * h + 1][w], 0x5140) ^ 0x80808080u;
              x[h][1] = __byte_perm(vw[j][2 * h][w], vw[j][2 * h + 1][w], 0x7362) ^ 0x80808080u;
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t sel = t & 1 ? 0x4342 : 0x4140;
              const uint32_t b0 = half2_of_codes(x[0][t / 2], sel), b1 = half2_of_codes(x[1][t / 2], sel);
#pragma unroll
              for (int m = 0; m < MT; ++m) mma16816(o[m][t], pa[m][j], b0, b1);
            }
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              float2& to = sum[m][COLS * dc + 4 * w + t];
              to = __ffma2_rn(make_float2(vs, vs),
                              __fadd2_rn(make_float2(o[m][t][0], o[m][t][1]), make_float2(o[m][t][2], o[m][t][3])), to);
            }
        }
      }
    }
    __syncwarp();  // every lane is done with the ring

    if (ue >= u_end) grid_launch_dependents();
    // ---- the next piece begins while the warps' sums of this one are added up, in order
    const bool whole = u <= first && ue == seg_end;
    const int done_np = np, done_g = g, done_p0 = p0;
    const Kv8Span done = span;
    const size_t slot = (size_t)(2 * blockIdx.x + (u_begin > first ? 0 : 1)) * S::PAIRS;
    u = ue;
    more = begin();
    auto merge = [&](int w, int m) {  // warp w's [8][D] of M tile m
      return reinterpret_cast<float*>(smem + (m == 0 ? (w * S::SLOTS + S::SLOTS - 1) * S::SLOT : S::OFF_M + w * S::SLOT));
    };
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      l[m] += __shfl_xor_sync(0xffffffffu, l[m], 1);
      l[m] += __shfl_xor_sync(0xffffffffu, l[m], 2);
      if (c == 0) s_ml[warp][8 * m + r] = make_float2(ref[m] == -INFINITY ? -INFINITY : ref[m] - HEADROOM, l[m]);
      float* to = merge(warp, m) + r * D;
      constexpr int COLS = D >= 128 ? 16 : 8;
#pragma unroll
      for (int dc = 0; dc < (D + 127) / 128; ++dc)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < COLS; i += 4) {
            const float2* f = sum[m] + COLS * dc + i;
            *reinterpret_cast<float4*>(to + 128 * dc + (2 * c + h) * COLS + i) =
                h ? make_float4(f[0].y, f[1].y, f[2].y, f[3].y) : make_float4(f[0].x, f[1].x, f[2].x, f[3].x);
          }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < done_np * (D / 4); i += THREADS) {
      const int p = i / (D / 4), d = 4 * (i % (D / 4));
      float m = -INFINITY, all = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) m = fmaxf(m, s_ml[w][p].x);
      if (m == -INFINITY) m = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 ml = s_ml[w][p];
        const float f = piece_factor(ml, m);
        const float4 y = *reinterpret_cast<const float4*>(merge(w, p / 8) + (p % 8) * D + d);
        all = fmaf(f, ml.y, all);
        o = make_float4(fmaf(f, y.x, o.x), fmaf(f, y.y, o.y), fmaf(f, y.z, o.z), fmaf(f, y.w, o.w));
      }
      if (whole) {
        finish4(a, done.r0, done.n, done_g, done_p0 + p, D, d, o, m, all);
      } else {
        if (d == 0) a.part_ml[slot + p] = make_float2(m, all);
        *reinterpret_cast<float4*>(a.part_o + (slot + p) * D + d) = o;
      }
    }
    // (the next fragments are written, and synchronised on, before these slots are sent into again)
  }
}

// Of which CTAs a segment has pieces: c0 and how many from there on. The first
// wrote its piece as the segment that it began, the others as the one that they
// continued.
struct Pieces {
  int c0, n;
  __device__ __forceinline__ size_t slot(const AttnArgs& a, int i, int pair) const {
    return (size_t)(2 * (c0 + i) + (i == 0)) * a.pairs + pair % a.pairs;
  }
};
template <int D>
__device__ __forceinline__ Pieces pieces_of(const AttnArgs& a, int total, int seq_u0, int su, int g, int pair) {
  if (a.whole) return Pieces{0, 1};
  const int u0 = seq_u0 + (pair / a.pairs * a.v.kv_heads + g) * su, ctas = sharing_ctas(a, total);
  const int c0 = cta_of(u0 + overhead_units(D), ctas, total);
  const int n = cta_of(u0 + su - 1, ctas, total) - c0 + 1;
  return c0 >= 0 && n > 0 && c0 + n <= a.ctas ? Pieces{c0, n} : Pieces{0, 1};  // (lengths that changed meanwhile)
}

// The combination's CTAs, blockIdx.x < combine_x: one for each (row, head) pair
// of the call, numbered through over the grid's rows, whichever sequence it is of
// (a grid of the most rows by all sequences has as many times more CTAs as the
// batch is ragged: 256 sequences of 2 rows and 32 heads with max_rows left out,
// 4 million for 16384 pairs). D / 4 threads take four dims each of every
// GROUPS-th of its pieces, so that the loads are under way at once, then add up. The
// weights' CTAs behind them, for sequence blockIdx.y: each 4 positions a thread of
// a KV head; 8 threads find the maximum and total of a pair from its pieces' anew,
// 64 pairs at a time, and each thread adds up its positions' weights in the pairs'
// order.
constexpr int W_PAIRS = 64;

template <int D, int GROUPS>
__global__ void __launch_bounds__(D / 4 * GROUPS) kv8_finish_kernel(const __grid_constant__ AttnArgs a, int combine_x) {
  constexpr int LANES = D / 4, THREADS = LANES * GROUPS;
  __shared__ float4 s_o[GROUPS][LANES];
  __shared__ float2 s_ml[GROUPS > W_PAIRS ? GROUPS : W_PAIRS];
  const Kv8View& v = a.v;
  const bool combines = (int)blockIdx.x < combine_x;
  const int unit = (int)(blockIdx.y * combine_x + blockIdx.x), row = unit / a.heads, head = unit % a.heads;
  grid_dependency_wait();
  grid_launch_dependents();
  if (combines && row >= v.num_rows) return;
  const int b = combines ? kv8_sequence_of(v, row) : (int)blockIdx.y, len = kv8_len(v, b), su = segment_units(a, len);
  const Kv8Span span = kv8_rows(v, b);
  const int total = a.prefix[v.num_seqs], seq_u0 = a.prefix[b];
  const int pairs = total > 0 ? span.n * a.group : 0;  // of a KV head

  if (combines) {
    const int g = head / a.group, pair = (row - span.r0) * a.group + head % a.group;
    if (pair < 0 || pair >= pairs) return;
    const Pieces pieces = pieces_of<D>(a, total, seq_u0, su, g, pair);
    if (pieces.n == 1) return;
    const int group = threadIdx.x / LANES, d = 4 * (threadIdx.x % LANES);
    float m = -INFINITY, all = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto take = [&](float2 ml, const float4& x) {  // the reference follows the largest so far
      const float now = ml.y > 0.f ? fmaxf(m, ml.x) : m;
      const float keep = m == now ? 1.f : exp2f(m - now), f = piece_factor(ml, now);
      m = now;
      all = fmaf(f, ml.y, all * keep);
      o = make_float4(fmaf(f, x.x, o.x * keep), fmaf(f, x.y, o.y * keep), fmaf(f, x.z, o.z * keep),
                      fmaf(f, x.w, o.w * keep));
    };
#pragma unroll 8
    for (int i = group; i < pieces.n; i += GROUPS) {
      const size_t slot = pieces.slot(a, i, pair);
      take(a.part_ml[slot], *reinterpret_cast<const float4*>(a.part_o + slot * D + d));
    }
    s_o[group][threadIdx.x % LANES] = o;
    if (threadIdx.x % LANES == 0) s_ml[group] = make_float2(m, all);
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) take(s_ml[i], s_o[i][threadIdx.x]);
    finish4(a, span.r0, span.n, g, pair, D, d, o, m == -INFINITY ? 0.f : m, all);
    return;
  }

  // ---- w_j
  const int g = (int)((blockIdx.x - combine_x) % v.kv_heads);
  const long long j0 = (long long)((blockIdx.x - combine_x) / v.kv_heads) * (4 * THREADS);
  if (a.accumulate && j0 >= len) return;
  const long long j = j0 + 4 * (int)threadIdx.x;
  const int lane = threadIdx.x & 7;  // of the 8 that look at a pair's pieces
  const size_t at = pair_at(a, span.r0, span.n, g);
  const float* scores = a.scores + at * a.scores_ld + j;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (j0 < len) {
    for (int p0 = 0; p0 < pairs; p0 += W_PAIRS) {
      const int np = min(W_PAIRS, pairs - p0);
      __syncthreads();
      for (int p = threadIdx.x / 8; p < (np + 3) / 4 * 4; p += THREADS / 8) {  // (whole warps)
        const Pieces pieces = pieces_of<D>(a, total, seq_u0, su, g, p0 + min(p, np - 1));
        float m = -INFINITY, all = 0.f;
        if (pieces.n > 1) {
#pragma unroll 4
          for (int i = lane; i < pieces.n; i += 8) {
            const float2 ml = a.part_ml[pieces.slot(a, i, p0 + min(p, np - 1))];
            const float now = ml.y > 0.f ? fmaxf(m, ml.x) : m;
            all = fmaf(piece_factor(ml, now), ml.y, all * (m == now ? 1.f : exp2f(m - now)));
            m = now;
          }
        }
        float top = m;
#pragma unroll
        for (int x = 4; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        all = m == -INFINITY ? all : all * exp2f(m - top);  // (a lane without pieces: 0, or NaN)
#pragma unroll
        for (int x = 4; x > 0; x >>= 1) all += __shfl_xor_sync(0xffffffffu, all, x);
        if (lane == 0 && p < np) {
          const float2 ml = pieces.n == 1 ? a.final_ml[at + p0 + p]
                                          : make_float2(top == -INFINITY ? 0.f : top, all > 0.f || all != all ? 1.f / all : 0.f);
          // Where the total is NaN, a reference that leaves a NaN score NaN and turns that of
          // a position behind the row, minus infinity, into the weight 0 (minus infinity less
          // NaN would be NaN).
          s_ml[p] = ml.y != ml.y ? make_float2(INFINITY, 1.f) : ml;
        }
      }
      __syncthreads();
      if (j < len) {
#pragma unroll 8
        for (int p = 0; p < np; ++p) {
          const float2 ml = s_ml[p];
          const float4 s = __ldcs(reinterpret_cast<const float4*>(scores + (size_t)(p0 + p) * a.scores_ld));
          sum[0] = fmaf(exp2_fast(s.x - ml.x), ml.y, sum[0]);
          sum[1] = fmaf(exp2_fast(s.y - ml.x), ml.y, sum[1]);
          sum[2] = fmaf(exp2_fast(s.z - ml.x), ml.y, sum[2]);
          sum[3] = fmaf(exp2_fast(s.w - ml.x), ml.y, sum[3]);
        }
      }
    }
  }
  float* w = a.weights + ((size_t)b * v.kv_heads + g) * a.weights_ld + j;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (j + t >= a.weights_ld || (a.accumulate && j + t >= len)) break;
    float x = j + t < len ? sum[t] : 0.f;
    if (a.accumulate && j + t < len - span.n) x += w[t];
    w[t] = x;
  }
}

struct Layout {
  int mt, ctas;
  size_t prefix, part_ml, part_o, final_ml, scores, bytes;
};

int scores_ld(const Kv8View& v) { return (int)(((long long)v.max_len + TILE - 1) / TILE * TILE); }

Layout layout_of(const Kv8View& v, const Kv8Attention& a) {
  Layout l;
  const int group = a.heads / v.kv_heads;
  l.mt = m_tiles(v.dim, (long long)a.tile_rows * group);
  const int pairs = 8 * l.mt, most_ctas = ctas_per_sm(v.dim, l.mt) * num_sms();  // those that run at once
  const long long segs = ((long long)v.num_rows * group / pairs + v.num_seqs) * v.kv_heads;  // at most
  const long long most = segs * (v.max_len / UNIT + 1 + overhead_units(v.dim));
  l.ctas = (int)(most < most_ctas ? most : most_ctas);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
  };
  l.prefix = take(((size_t)v.num_seqs + 1) * 4);
  l.part_ml = take((size_t)2 * l.ctas * pairs * 8);
  l.part_o = take((size_t)2 * l.ctas * pairs * v.dim * 4);
  l.final_ml = take(a.weights ? (size_t)v.num_rows * a.heads * 8 : 0);
  l.scores = take(a.weights ? (size_t)v.num_rows * a.heads * scores_ld(v) * 4 : 0);
  l.bytes = at;
  return l;
}

template <int D, int GROUPS>
cudaError_t launch_finish(const AttnArgs& a, cudaLaunchConfig_t cfg) {
  constexpr int N = D / 4 * GROUPS;
  const long long pairs = (long long)a.v.num_rows * a.heads;  // (below 2^30: the arguments are checked for the units they make)
  const long long combine = a.whole ? 0 : (pairs + a.v.num_seqs - 1) / a.v.num_seqs;
  const long long span = a.weights ? (a.accumulate ? a.v.max_len : a.weights_ld) : 0;
  const long long ctas = combine + (span + 4 * N - 1) / (4 * N) * a.v.kv_heads;
  if (ctas == 0) return cudaSuccess;  // weights added up over tables of no pages
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)a.v.num_seqs);
  cfg.blockDim = dim3(N);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv8_finish_kernel<D, GROUPS>, a, (int)combine);
}

template <int D, int MT>
cudaError_t launch_shape(const AttnArgs& a, cudaStream_t s) {
  using S = Shape<D, MT>;
  static bool ready[64] = {};  // the attribute is set once for each device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(kv8_attention_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = S::BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv8_attention_kernel<D, MT>, a);
  if (e != cudaSuccess || (a.whole && !a.weights)) return e;
  // few (row, head) pairs have many pieces each; of many pairs most are whole or in two pieces
  return (long long)a.v.num_rows * a.heads <= 4 * num_sms() ? launch_finish<D, 8>(a, cfg) : launch_finish<D, 2>(a, cfg);
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
  a.pairs = 8 * l.mt;
  a.scale_log2 = in.scale * 1.4426950408889634f;
  a.ctas = l.ctas;
  const bool one_segment = (long long)in.tile_rows * a.group <= a.pairs;  // of a KV head
  a.whole = (long long)v.max_len * v.dim <= (in.weights && one_segment && v.dim < 256 ? WHOLE_SIZE_WEIGHTED : WHOLE_SIZE);
  a.prefix = reinterpret_cast<int*>(base + l.prefix);
  a.part_ml = reinterpret_cast<float2*>(base + l.part_ml);
  a.part_o = reinterpret_cast<float*>(base + l.part_o);
  if (in.weights) {
    a.final_ml = reinterpret_cast<float2*>(base + l.final_ml);
    a.scores = reinterpret_cast<float*>(base + l.scores);
    a.scores_ld = scores_ld(v);
    a.weights = in.weights;
    a.weights_ld = in.weights_ld;
    a.accumulate = in.accumulate;
  }
  if (v.dim == 256) return launch_shape<256, 1>(a, s);
  if (v.dim == 128) return l.mt == 1 ? launch_shape<128, 1>(a, s) : launch_shape<128, 2>(a, s);
  return l.mt == 1 ? launch_shape<64, 1>(a, s) : launch_shape<64, 2>(a, s);
}

}  // namespace apr
