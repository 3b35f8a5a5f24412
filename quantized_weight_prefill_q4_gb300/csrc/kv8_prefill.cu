// Attention of chunks of rows over their sequences' 8-bit paged KV caches
// (include/apr_kv8.h): for each (row, head) pair
//   p_j = softmax_j(scale q . (c_j s)),  out = sum_j p_j (c'_j s'),  j <= its position
//
// Bound. 4 D operations a pair and position, and every code is read once for 128 or 256
// pairs, so the tensor cores bound it: M = 128 pairs of one KV head a tile, keys in
// tiles of KT. Both products take fp16: codes are exact in it, a page's
// scale is a factor of 32 or more neighbouring scores (K) or weights (V).
//
// Segments. A segment is MT * 128 (row, head) pairs of a sequence that read one KV head,
// over all positions that its last row sees. What segments cost (positions, and a start
// worth START of them) is numbered through, a sequence's as a quadratic in closed form, and each CTA takes an
// equal, contiguous share: chunks of any lengths in one batch keep every SM equally busy. A
// segment within one share is finished there; of the others each CTA that has a piece
// writes its outputs, reference maximum and total, and a second kernel combines them in order.
//
// A CTA. The roles hand work to each other through mbarriers:
//   softmax    four warps for each M tile, a thread a pair (tensor memory lane): they
//              write q into shared memory, then per key tile read the scores, move the
//              running maximum and sum, and write the weights
//              into tensor memory; O is rescaled only when a maximum grows by more than 2^MOVE
//   converters turn codes into fp16 tiles in a ring of slots, rows of 128 bytes
//              swizzled for the tensor cores: as they lie in memory for K (dims contiguous, the
//              product's k side) and for V (dims contiguous, the N side)
//   one warp   issues S = Q K^T (both from shared memory) and O += P V (P from tensor memory)
// With two M tiles the tensor cores work on one while the other's softmax runs; with
// one (256 dims) on the next key tile's scores.
//
// float32 rows: q and the weights enter as two fp16 pieces each (22 bits), twice the
// products. The tensor cores' sums lose about 2e-8 of themselves at each step, so O is
// taken over into a float32 mean every FOLD positions.
//
// Weights. A pair's weights are 2^7 p v, p against a reference at most MOVE (base 2) below the
// maximum, v the page's V scale over a power of two R that no scale so far exceeds: at most 2^15.

#include "apr_internal.h"
#include "host_common.h"
#include "kv8.cuh"

namespace apr {
namespace {

constexpr int START = 256;       // positions that a segment's start and end are worth
constexpr int MIN_TILES = 2;     // of a CTA's share
constexpr float MOVE = 8.f;
constexpr int FOLD = 512;        // positions
constexpr int SOFT_WARPS = 8, CONV_WARPS = 4, MMA_WARP = SOFT_WARPS + CONV_WARPS;  // (one M tile: 4 and 8)
constexpr int THREADS = 32 * (MMA_WARP + 1);

struct PrefillArgs {
  Kv8View v;
  const void* q;
  void* out;
  long long ldq, ldo;
  int heads, group;
  float scale_log2;  // softmax scale times log2(e)
  int ctas;          // of the grid
  int4* record;      // [ctas] (sequence, segment of it, KV head, pieces) of the segment that a CTA begins and others end
  float2* part_ml;   // [2 ctas][pairs] reference maximum and total of a piece
  float4* part_o;    // [2 ctas][D / 4][pairs] its outputs
  float4* mean;      // [ctas][D / 4][pairs] the mean taken over (float32 rows)
};

template <int D_, bool TWO_>
struct Shape {
  static constexpr int D = D_;
  static constexpr bool TWO = TWO_;                        // two fp16 pieces of q and of the weights
  static constexpr int MT = D <= 128 ? 2 : 1;              // M tiles
  static constexpr int PAIRS = 128 * MT;
  static constexpr int KT = D <= 128 && !TWO ? 128 : 64;   // keys of a tile
  static constexpr int GROUPS = KT / 32;                   // of 32 positions, within one page each
  static constexpr int PIECES = TWO ? 2 : 1;
  static constexpr int PANEL = KT * 128;                   // bytes of 64 dims of a tile
  static constexpr int SLOT = KT * D * 2;
  static constexpr int Q_BYTES = MT * PIECES * 128 * D * 2;
  static constexpr int SLOTS_FIT = (226 * 1024 - Q_BYTES) / SLOT;
  static constexpr int SLOTS = SLOTS_FIT < 6 ? SLOTS_FIT : 6;
  static constexpr int SMEM = Q_BYTES + SLOTS * SLOT + 1024;
  static constexpr int SOFT = 4 * MT, CONV = MMA_WARP - SOFT;  // warps
  static constexpr int EACH = KT * D / 16 / (32 * CONV);   // 16-byte pieces of a chunk that a converter thread has
  // tensor memory columns: O of each M tile, then two buffers of scores, then (where there is room) two of weights
  static constexpr int COL_S = MT * D;
  static constexpr int P_COLS = PIECES * KT / 2;
  static constexpr bool OWN_P = COL_S + 2 * KT + 2 * P_COLS <= 512;
  static constexpr int COL_P = OWN_P ? COL_S + 2 * KT : COL_S;
  static constexpr int P_STEP = OWN_P ? P_COLS : KT;
  static_assert(COL_S + 2 * KT <= 512 && (OWN_P || !TWO), "tensor memory");
  static_assert(SLOTS >= 3 && SMEM + 2048 <= 232448, "shared memory");
  static_assert(EACH >= 1 && KT * D / 16 % (32 * CONV) == 0, "converters");
  static constexpr int FOLD_TILES = FOLD / KT;
};

// ---------------------------------------------------------------- the work
// A sequence's segments: of `rows` rows at positions first .. len - 1.
struct Work {
  int len, first, r0, n;
  long long base, pairs;  // (START + what the first row sees) * group; (row, head) pairs of a KV head
  int segments;           // of a KV head
};
template <class S>
__device__ __forceinline__ Work work_of(const PrefillArgs& a, int b) {
  Work w;
  const Kv8Span span = kv8_rows(a.v, b);
  w.len = kv8_len(a.v, b);
  w.r0 = span.r0, w.n = span.n;
  w.first = w.len - w.n;
  w.base = (long long)(START + max(w.first, 0)) * a.group;
  w.pairs = (long long)w.n * a.group;
  w.segments = (int)((w.pairs + S::PAIRS - 1) / S::PAIRS);
  return w;
}
// What segment t of one KV head costs, in positions * group; segments 0 .. t - 1 (t < segments).
template <class S>
__device__ __forceinline__ long long cost(const Work& w, int t) {
  return w.base + min(w.pairs, (long long)(t + 1) * S::PAIRS);
}
template <class S>
__device__ __forceinline__ long long cost_before(const Work& w, int t) {
  return (long long)t * w.base + (long long)t * (t + 1) / 2 * S::PAIRS;
}
template <class S>
__device__ __forceinline__ long long cost_all(const PrefillArgs& a, const Work& w) {
  return w.segments == 0 ? 0 : a.v.kv_heads * (cost_before<S>(w, w.segments - 1) + cost<S>(w, w.segments - 1));
}
// Key tiles of segment t: those that its last pair's row sees, one at least.
template <class S>
__device__ __forceinline__ int key_tiles(const PrefillArgs& a, const Work& w, int t) {
  const long long last = min(w.pairs, (long long)(t + 1) * S::PAIRS) - 1;
  const int sees = w.first + (int)(last / a.group) + 1;
  return max(1, (sees + S::KT - 1) / S::KT);
}
// The key tile of a segment that a share begins with which begins `at` into the segment's cost.
template <class S>
__device__ __forceinline__ int tile_at(const PrefillArgs& a, long long at, int tiles) {
  const long long in = at - (long long)START * a.group, step = (long long)S::KT * a.group;
  return in <= 0 ? 0 : (int)min((long long)tiles, (in + step - 1) / step);
}
// Where CTA c's share of `total` begins, of `ctas`.
__device__ __forceinline__ long long share_begin(int c, int ctas, long long total) {
  return (long long)((unsigned long long)total / ctas) * c + (long long)((unsigned long long)total % ctas) * c / ctas;
}

struct Piece {
  Work w;
  int b, g, t;
  long long p0;
  int np;            // pairs of the segment
  int k0, k1;        // its key tiles k0 .. k1 - 1
  int tiles;         // of the segment
};

// The pieces of a CTA's share, one after the other; a whole warp calls it.
template <class S>
struct Pieces {
  int b, ctas;
  long long u, end, seq_u0, total;

  __device__ __forceinline__ bool next(const PrefillArgs& a, Piece& p) {
    const int lane = threadIdx.x & 31;
    while (u < end && b < a.v.num_seqs) {
      p.w = work_of<S>(a, b);
      const long long all = cost_all<S>(a, p.w);
      if (u >= seq_u0 + all) {  // the next sequence that has rows
        seq_u0 += all;
        ++b;
        for (;;) {
          const int mine = b + lane;
          const bool has = mine < a.v.num_seqs && kv8_rows(a.v, mine).n > 0;
          const unsigned m = __ballot_sync(0xffffffffu, has);
          if (m) {
            b += __ffs(m) - 1;
            break;
          }
          b += 32;
          if (b >= a.v.num_seqs) return false;
        }
        continue;
      }
      const long long at = u - seq_u0;
      int lo = 0, hi = p.w.segments;  // the last segment that begins at or before it
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (a.v.kv_heads * cost_before<S>(p.w, mid) <= at)
          lo = mid;
        else
          hi = mid;
      }
      const long long before = a.v.kv_heads * cost_before<S>(p.w, lo), one = cost<S>(p.w, lo);
      p.b = b;
      p.t = lo;
      p.g = (int)min((at - before) / one, (long long)a.v.kv_heads - 1);
      const long long seg_u0 = seq_u0 + before + p.g * one, seg_end = seg_u0 + one;
      p.tiles = key_tiles<S>(a, p.w, lo);
      p.k0 = u == seg_u0 ? 0 : tile_at<S>(a, u - seg_u0, p.tiles);
      p.k1 = end >= seg_end ? p.tiles : tile_at<S>(a, end - seg_u0, p.tiles);
      u = min(end, seg_end);
      if (p.k0 >= p.k1) continue;
      p.p0 = (long long)lo * S::PAIRS;
      p.np = (int)min((long long)S::PAIRS, p.w.pairs - p.p0);
      return true;
    }
    return false;
  }
  // Pieces of the segment that p begins (k0 == 0), this CTA the c-th.
  __device__ __forceinline__ int count(const PrefillArgs& a, const Piece& p, int c) const {
    const long long one = cost<S>(p.w, p.t), seg_u0 = seq_u0 + a.v.kv_heads * cost_before<S>(p.w, p.t) + p.g * one;
    int n = 1;
    for (++c; c < ctas; ++c, ++n) {
      const long long at = share_begin(c, ctas, total);
      if (at >= seg_u0 + one || tile_at<S>(a, at - seg_u0, p.tiles) >= p.tiles) break;
    }
    return n;
  }
};

// ---------------------------------------------------------------- pages
// What a warp knows of the pages of 64 neighbouring groups of 32 positions: a lane has a
// group's value, the next 32 groups' on their way.
template <typename V, typename F>
struct Window {
  V now, next;
  int base;
  __device__ __forceinline__ void begin(int group, const F& load) {
    base = group;
    now = load(group + (int)(threadIdx.x & 31));
    next = load(group + 32 + (int)(threadIdx.x & 31));
  }
  __device__ __forceinline__ void reach(int group, const F& load) {
    if (group - base < 32) return;
    base += 32;
    now = next;
    next = load(base + 32 + (int)(threadIdx.x & 31));
  }
};

// Where the codes of a group of 32 positions lie, in groups (page ids out of range read page 0, flagged).
__device__ __forceinline__ uint32_t group_at(const PrefillArgs& a, const Piece& p, int group) {
  if (group * 32ll >= p.w.len) return 0;
  const int pos = group * 32, page = max(kv8_page(a.v, p.b, pos >> a.v.page_shift), 0);
  return (uint32_t)(kv8_scale_at(a.v, page, p.g) << (a.v.page_shift - 5)) +
         (uint32_t)((pos >> 5) & ((1 << (a.v.page_shift - 5)) - 1));
}
__device__ __forceinline__ float2 group_scales(const PrefillArgs& a, const Piece& p, int group) {
  if (group * 32ll >= p.w.len) return make_float2(0.f, 0.f);
  const size_t at = kv8_scale_at(a.v, max(kv8_page(a.v, p.b, group * 32 >> a.v.page_shift), 0), p.g);
  return make_float2(a.v.k_scale[at], a.v.v_scale[at]);
}

// ---------------------------------------------------------------- tensor core operands
__device__ __forceinline__ void mma_f16_ss_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// V as the second product's B: N (dims) contiguous, 64 of them a 128-byte row, panels of 64 dims `panel`
// bytes apart (leading byte offset), groups of 8 positions 1024 (stride byte offset).
__device__ __forceinline__ uint64_t smem_desc_n_major(const void* tile, uint32_t panel) {
  return (smem_desc_sw128(tile) & ~((uint64_t)0x3fff << 16)) | (uint64_t)(panel >> 4) << 16;
}
constexpr uint32_t N_MAJOR_B = 1u << 16;

// 32 lanes x 16 columns, from v[0 .. 15].
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// ---------------------------------------------------------------- rows
template <typename T>
__device__ __forceinline__ void store4(T* p, const float4& x) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(p) = x;
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(x.x, x.y), pack2<T>(x.z, x.w));
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, 1) kv8_prefill_kernel(const __grid_constant__ PrefillArgs a) {
  using S = Shape<D, sizeof(T) == 4>;
  grid_dependency_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* ring = smem + S::Q_BYTES;
  __shared__ uint64_t full[S::SLOTS], empty[S::SLOTS], q_full[2], s_full[2], p_full[2], o_done[2], o_last[2], drain;
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_words[2];  // the second is never set: the drain's wait ignores the abort
  __shared__ long long s_scan[MMA_WARP + 1], s_found[1];
  __shared__ int s_found_b;
  volatile int* abort_flag = abort_words;
  const Kv8View& v = a.v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // ---- what the sequences cost, and where this CTA's share begins: a thread counts `run` neighbouring sequences
  const int run = (v.num_seqs + THREADS - 1) / THREADS;
  const int my_b0 = min((int)threadIdx.x * run, v.num_seqs), my_b1 = min(my_b0 + run, v.num_seqs);
  long long mine = 0;
  for (int b = my_b0; b < my_b1; ++b) mine += cost_all<S>(a, work_of<S>(a, b));
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_scan[warp] = inc;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::SLOTS; ++i) {
      mbar_init(&full[i], S::CONV);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_last[i], 1);
    }
    mbar_init(&drain, 1);
    abort_words[0] = abort_words[1] = 0;
    s_found_b = 0;
    s_found[0] = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) tmem_alloc(&tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  long long my_u0 = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w <= MMA_WARP; ++w) {
    if (w < warp) my_u0 += s_scan[w];
    total += s_scan[w];
  }
  Pieces<S> pieces;
  pieces.total = total;
  pieces.ctas = (int)max(1ll, min((long long)a.ctas, total / ((long long)MIN_TILES * S::KT * a.group)));
  const bool idle = (int)blockIdx.x >= pieces.ctas || total <= 0;
  pieces.u = idle ? 0 : share_begin(blockIdx.x, pieces.ctas, total);
  pieces.end = idle ? 0 : share_begin(blockIdx.x + 1, pieces.ctas, total);
  if (!idle && my_u0 <= pieces.u && pieces.u < my_u0 + mine) {
    int b = my_b0;
    long long at = my_u0;
    for (long long n; b + 1 < my_b1 && at + (n = cost_all<S>(a, work_of<S>(a, b))) <= pieces.u; ++b) at += n;
    s_found_b = b;
    s_found[0] = at;
  }
  __syncthreads();
  pieces.b = s_found_b;
  pieces.seq_u0 = s_found[0];
  Piece p;

  if (warp < S::SOFT) {
    // ------------------------------------------------ softmax
    const int m = warp / 4, r = (int)threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16), o_col = lanes + m * D;
    const T* q = static_cast<const T*>(a.q);
    T* out = static_cast<T*>(a.out);
    int cnt = 0, npiece = 0;  // key tiles and pieces so far
    bool ok = true, begun = false;
    auto wait = [&](uint64_t* bar, int phase) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(phase & 1), abort_flag, v.status));
      return ok;
    };
    auto scales_of = [&](int group) { return group_scales(a, p, group); };
    Window<float2, decltype(scales_of)> scales;
    while (ok && pieces.next(a, p)) {
      if (128 * m >= p.np) continue;
      // ---- the row: fp16 pieces times a power of two that brings the largest magnitude into [1, 2)
      scales.begin(p.k0 * S::GROUPS, scales_of);
      const bool live = 128 * m + r < p.np;
      const long long pair = p.p0 + 128 * m + (live ? r : 0);
      const int i = (int)(pair / a.group);
      const size_t head = (size_t)p.g * a.group + (size_t)(pair % a.group);
      const T* qr = q + (long long)(p.w.r0 + i) * a.ldq + head * D;
      float top = 0.f;
      bool odd = false;
#pragma unroll 8
      for (int d = 0; d < D; d += 8) {
        float x[8];
        values8(load8(qr + d), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e])), odd |= x[e] != x[e];
      }
      const int e2 = top <= FLT_MAX ? min(max((int)(__float_as_uint(top) >> 23) - 127, -120), 120) : 0;
      const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
      // (a NaN or an infinity: every score of the row NaN, its products finite)
      const bool bad = odd || !(top <= FLT_MAX);
      const float factor = bad ? __int_as_float(0x7fffffff) : a.scale_log2 * __uint_as_float((uint32_t)(127 + e2) << 23);
      uint8_t* sq = sQ + m * S::PIECES * 128 * D * 2 + r * 128;
#pragma unroll 4
      for (int d = 0; d < D; d += 8) {
        float x[8];
        values8(load8(qr + d), x);
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y0 = live && !bad ? x[2 * e] * down : 0.f, y1 = live && !bad ? x[2 * e + 1] * down : 0.f;
          h[e] = half2_bits(y0, y1);
          const float2 f = half2_values(h[e]);
          l[e] = half2_bits(y0 - f.x, y1 - f.y);
        }
        uint8_t* to = sq + (d / 64) * 128 * 128 + (((d / 8 % 8) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
        if constexpr (S::TWO) *reinterpret_cast<uint4*>(to + 128 * D * 2) = make_uint4(l[0], l[1], l[2], l[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[m]);
      ++npiece;

      const int sees = live ? min(p.w.len, p.w.first + i + 1) : 0;  // positions
      float ref = -INFINITY, run_max = -INFINITY, sum = 0.f;
      float R = 0x1p-100f, inv_R = 0x1p100f;
      float mean_ref = -INFINITY, mean_sum = 0.f;  // of the mean taken over
      const bool partial = p.k1 - p.k0 < p.tiles;
      const int slot = 2 * (int)blockIdx.x + (p.k0 == 0);
      // ---- O, with the mean taken over so far, to the mean, a piece's outputs or the rows
      auto flush = [&](bool last) {
        const float top_ref = fmaxf(ref, mean_ref);
        const float wn = sum == 0.f ? 0.f : exp2f(ref - top_ref), wm = mean_sum == 0.f ? 0.f : exp2f(mean_ref - top_ref);
        const float all = sum * wn + mean_sum * wm, inv = all == 0.f ? 0.f : 1.f / all;
        const float co = R * 0x1p-7f * (wn * inv), cm = wm * mean_sum * inv;
        float4* mean = a.mean + (size_t)blockIdx.x * (D / 4) * S::PAIRS + 128 * m + r;
        float4* part = a.part_o + (size_t)slot * (D / 4) * S::PAIRS + 128 * m + r;
        T* to = out + (long long)(p.w.r0 + i) * a.ldo + head * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(o_col + 32 * c, o);
          tmem_ld_wait_regs(o);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float4 y = make_float4(__uint_as_float(o[4 * k]) * co, __uint_as_float(o[4 * k + 1]) * co,
                                   __uint_as_float(o[4 * k + 2]) * co, __uint_as_float(o[4 * k + 3]) * co);
            const size_t at = (size_t)(8 * c + k) * S::PAIRS;
            if constexpr (S::TWO)
              if (mean_sum != 0.f) {
                const float4 x = mean[at];
                y.x = fmaf(x.x, cm, y.x), y.y = fmaf(x.y, cm, y.y), y.z = fmaf(x.z, cm, y.z), y.w = fmaf(x.w, cm, y.w);
              }
            if (all == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);  // (whatever O held)
            if (!last)
              mean[at] = y;
            else if (partial)
              part[at] = y;
            else if (live)
              store4<T>(to + 32 * c + 4 * k, y);
          }
        }
        mean_ref = top_ref;
        mean_sum = all;
        sum = 0.f;
      };
      bool fresh = true;  // O holds nothing yet
#pragma unroll 1
      for (int j = p.k0; j < p.k1; ++j, ++cnt) {
        const int buf = S::MT == 2 ? m : cnt & 1, phase = S::MT == 2 ? cnt : cnt >> 1;
        scales.reach(j * S::GROUPS, scales_of);
        float ks[S::GROUPS], vs[S::GROUPS];
        float vmax = 0.f;
#pragma unroll
        for (int c = 0; c < S::GROUPS; ++c) {
          ks[c] = __shfl_sync(0xffffffffu, scales.now.x, j * S::GROUPS + c - scales.base) * factor;
          vs[c] = __shfl_sync(0xffffffffu, scales.now.y, j * S::GROUPS + c - scales.base);
          vmax = fmaxf(vmax, vs[c]);
        }
        // (these scores' completion covers every product before them, O's of two tiles ago among them: so a wait for the
        // last tile's O, by parity, cannot be a phase behind)
        if (!wait(&s_full[buf], phase)) break;
        tc_fence_after();
        if (S::TWO && j > p.k0 && (j - p.k0) % S::FOLD_TILES == 0) {
          if (!wait(&o_done[m], cnt - 1)) break;
          tc_fence_after();
          flush(false);
          fresh = true;
        }
        const uint32_t s_col = lanes + S::COL_S + buf * S::KT, p_col = lanes + S::COL_P + buf * S::P_STEP;
        const int left = sees - j * S::KT;  // positions of the tile that the row sees
        const bool whole = __all_sync(0xffffffffu, left >= S::KT);
        float tile_max = -INFINITY;
#pragma unroll
        for (int c = 0; c < S::GROUPS; ++c) {
          uint32_t s[32];
          tmem_ld_32x32b_x32(s_col + 32 * c, s);
          tmem_ld_wait_regs(s);
          float x[2] = {-INFINITY, -INFINITY};
          if (whole) {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k & 1] = fmaxf(x[k & 1], __uint_as_float(s[k]));
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k & 1] = 32 * c + k < left ? fmaxf(x[k & 1], __uint_as_float(s[k])) : x[k & 1];
          }
          const float y = fmaxf(x[0], x[1]);
          tile_max = fmaxf(tile_max, y == -INFINITY ? y : y * ks[c]);
        }
        run_max = fmaxf(run_max, tile_max);
        // ---- the reference, and R: O moves with them
        const bool grow = vmax > R;
        if (fresh) {
          ref = run_max == -INFINITY ? 0.f : run_max;
          if (grow) {
            R = __uint_as_float(min((__float_as_uint(vmax) & 0x7f800000u) + (2u << 23), 0x7e800000u));
            inv_R = 1.f / R;
          }
        } else if (grow || __any_sync(0xffffffffu, run_max > ref + MOVE)) {
          if (!wait(&o_done[m], cnt - 1)) break;
          tc_fence_after();
          const float new_ref = run_max > ref ? run_max : ref;
          float f = exp2f(ref - new_ref);
          sum *= f;
          ref = new_ref;
          if (grow) {
            const float new_R = __uint_as_float(min((__float_as_uint(vmax) & 0x7f800000u) + (2u << 23), 0x7e800000u));
            f *= R * (1.f / new_R);
            R = new_R;
            inv_R = 1.f / R;
          }
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(o_col + 32 * c, o);
            tmem_ld_wait_regs(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st_32x32b_x32(o_col + 32 * c, o);
            tmem_st_wait();
          }
        }
        // ---- the weights
        float l[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < S::GROUPS; ++c) {
          uint32_t s[32];
          tmem_ld_32x32b_x32(s_col + 32 * c, s);
          tmem_ld_wait_regs(s);
          const float w = vs[c] * inv_R * 0x1p7f;
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float x0 = exp2_fast(fmaf(__uint_as_float(s[2 * k]), ks[c], -ref));
            float x1 = exp2_fast(fmaf(__uint_as_float(s[2 * k + 1]), ks[c], -ref));
            if (!whole) {
              x0 = 32 * c + 2 * k < left ? x0 : 0.f;
              x1 = 32 * c + 2 * k + 1 < left ? x1 : 0.f;
            }
            l[0] += x0, l[1] += x1;
            x0 *= w, x1 *= w;
            hi[k] = half2_bits(x0, x1);
            if constexpr (S::TWO) {
              const float2 f = half2_values(hi[k]);
              lo[k] = half2_bits(x0 - f.x, x1 - f.y);
            }
          }
          tmem_st_32x32b_x16(p_col + 16 * c, hi);
          if constexpr (S::TWO) tmem_st_32x32b_x16(p_col + S::KT / 2 + 16 * c, lo);
          tmem_st_wait();
        }
        sum += l[0] + l[1];
        fresh = false;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      if (!ok || !wait(&o_last[m], npiece - 1)) break;
      tc_fence_after();
      flush(true);
      tc_fence_before();
      if (partial) {
        a.part_ml[(size_t)slot * S::PAIRS + 128 * m + r] = make_float2(mean_ref, mean_sum);
        if (p.k0 == 0 && threadIdx.x == 0) {
          a.record[blockIdx.x] = make_int4(p.b, p.t, p.g, pieces.count(a, p, blockIdx.x));
          begun = true;
        }
      }
    }
    if (threadIdx.x == 0 && !begun) a.record[blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (warp < MMA_WARP) {
    // ------------------------------------------------ converters: chunks of K and V in the order in which they are used
    const int tid = (int)threadIdx.x - 32 * S::SOFT;
    constexpr int ROW = D / 16;                       // 16-byte pieces of a position's codes
    constexpr int STEP = 32 * S::CONV / ROW;          // positions from one of a thread's pieces to the next
    const int key0 = tid / ROW, piece = tid % ROW, panel = piece / 4;
    int done = 0;  // chunks so far
    bool ok = true;
    auto at_of = [&](int group) { return group_at(a, p, group); };
    Window<uint32_t, decltype(at_of)> at[2];
    while (ok && pieces.next(a, p)) {
      const int n = p.k1 - p.k0;
      at[0].begin(p.k0 * S::GROUPS, at_of);
      at[1] = at[0];
      uint4 w[2][S::EACH];
      // chunk c: K of tile 0, V of tile 0, K of tile 1, ..., or with one M tile K of tiles 0 and 1, V of tile 0, K of tile 2, ...
      auto load = [&](int c, uint4 (&x)[S::EACH]) {
        int j = c / 2, is_v = c & 1;
        if (S::MT == 1 && c > 0 && c < 2 * n - 1) is_v = !(c & 1), j = is_v ? (c - 2) / 2 : (c + 1) / 2;
        const int tile = p.k0 + j;
        at[is_v].reach(tile * S::GROUPS, at_of);
        const int8_t* codes = (is_v ? v.V : v.K) + piece * 16;
#pragma unroll
        for (int i = 0; i < S::EACH; ++i) {
          const int key = key0 + i * STEP;
          const uint32_t g = __shfl_sync(0xffffffffu, at[is_v].now, tile * S::GROUPS + key / 32 - at[is_v].base);
          x[i] = make_uint4(0, 0, 0, 0);
          if (tile * S::KT + key < p.w.len)
            x[i] = *reinterpret_cast<const uint4*>(codes + ((size_t)g * 32 + key % 32) * D);
        }
      };
      auto put = [&](const uint4 (&x)[S::EACH]) {
        const int s = done % S::SLOTS;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], (uint32_t)((done / S::SLOTS + 1) & 1), abort_flag, v.status));
        if (!ok) return;
        uint8_t* slot = ring + s * S::SLOT + panel * S::PANEL;
#pragma unroll
        for (int i = 0; i < S::EACH; ++i) {
          const int key = key0 + i * STEP;
          const uint32_t b[4] = {x[i].x ^ 0x80808080u, x[i].y ^ 0x80808080u, x[i].z ^ 0x80808080u, x[i].w ^ 0x80808080u};
          uint4 y[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            y[h] = make_uint4(half2_of_codes(b[2 * h], 0x4140), half2_of_codes(b[2 * h], 0x4342),
                              half2_of_codes(b[2 * h + 1], 0x4140), half2_of_codes(b[2 * h + 1], 0x4342));
          uint8_t* row = slot + key * 128;
          const int c = 2 * (piece & 3), odd = panel & 1;  // (neighbouring panels' stores go to different banks)
          *reinterpret_cast<uint4*>(row + (((c + odd) ^ (key & 7)) << 4)) = y[odd];
          *reinterpret_cast<uint4*>(row + (((c + 1 - odd) ^ (key & 7)) << 4)) = y[1 - odd];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        ++done;
      };
      load(0, w[0]);
#pragma unroll 1
      for (int c = 0; c < 2 * n && ok; c += 2) {
        load(c + 1, w[1]);
        put(w[0]);
        if (!ok) break;
        if (c + 2 < 2 * n) load(c + 2, w[0]);
        put(w[1]);
      }
    }
  } else {
    // ------------------------------------------------ the products
    constexpr uint32_t IDESC_S = idesc_f16_f32(128, S::KT), IDESC_O = idesc_f16_f32(128, D) | N_MAJOR_B;
    int chunks = 0, cnt[2] = {0, 0}, npiece[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(phase & 1), abort_flag, v.status));
      return ok;
    };
    while (ok && pieces.next(a, p)) {
      const int n = p.k1 - p.k0, nm = S::MT == 2 && p.np > 128 ? 2 : 1;
      auto k_chunk = [&](int j) { return chunks + (S::MT == 2 || j == 0 ? 2 * j : 2 * j - 1); };
      auto v_chunk = [&](int j) { return chunks + (S::MT == 2 || j == n - 1 ? 2 * j + 1 : 2 * j + 2); };
      auto issue_s = [&](int j, int m) {
        const int c = k_chunk(j), x = cnt[m] + j, buf = S::MT == 2 ? m : x & 1;
        if (!wait(&full[c % S::SLOTS], c / S::SLOTS)) return;
        tc_fence_after();
        const uint8_t* kt = ring + c % S::SLOTS * S::SLOT;
#pragma unroll
        for (int s = S::PIECES - 1; s >= 0; --s) {  // the small piece first
          const uint64_t qd = smem_desc_sw128(sQ + (m * S::PIECES + s) * 128 * D * 2), kd = smem_desc_sw128(kt);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_f16_ss_elect(tmem + S::COL_S + buf * S::KT, qd + (uint64_t)((kk / 4 * 128 * 128) >> 4) + 2 * (kk % 4),
                             kd + (uint64_t)((kk / 4 * S::PANEL) >> 4) + 2 * (kk % 4), IDESC_S, s != S::PIECES - 1 || kk != 0);
        }
        mma_commit_elect(&s_full[buf]);
        if (m == nm - 1) mma_commit_elect(&empty[c % S::SLOTS]);
      };
      auto issue_o = [&](int j, int m) {
        const int c = v_chunk(j), x = cnt[m] + j, buf = S::MT == 2 ? m : x & 1;
        if (!wait(&full[c % S::SLOTS], c / S::SLOTS)) return;
        if (!wait(&p_full[buf], S::MT == 2 ? x : x >> 1)) return;
        tc_fence_after();
        const uint8_t* vt = ring + c % S::SLOTS * S::SLOT;
        const bool fresh = S::TWO ? j % S::FOLD_TILES == 0 : j == 0;
#pragma unroll
        for (int s = S::PIECES - 1; s >= 0; --s) {
          const uint64_t vd = smem_desc_n_major(vt, S::PANEL);
#pragma unroll
          for (int kk = 0; kk < S::KT / 16; ++kk)
            mma_f16_ts_elect(tmem + m * D, tmem + S::COL_P + buf * S::P_STEP + s * (S::KT / 2) + 8 * kk, vd + (uint64_t)((kk * 2048) >> 4),
                             IDESC_O, !fresh || s != S::PIECES - 1 || kk != 0);
        }
        mma_commit_elect(&o_done[m]);
        if (j == n - 1) mma_commit_elect(&o_last[m]);
        if (m == nm - 1) mma_commit_elect(&empty[c % S::SLOTS]);
      };
      for (int m = 0; m < nm && ok; ++m) {
        wait(&q_full[m], npiece[m]);
        if (ok) issue_s(0, m);
      }
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j) {
        if (S::MT == 2) {
          for (int m = 0; m < nm && ok; ++m) {
            issue_o(j, m);
            if (ok && j + 1 < n) issue_s(j + 1, m);
          }
        } else {
          if (j + 1 < n) issue_s(j + 1, 0);
          if (ok) issue_o(j, 0);
        }
      }
      for (int m = 0; m < nm; ++m) cnt[m] += n, ++npiece[m];
      chunks += 2 * n;
    }
    // the products in flight have finished before tensor memory goes
    mma_commit_elect(&drain);
    __all_sync(0xffffffffu, mbar_wait(&drain, 0, abort_flag + 1, v.status));
  }
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- the pieces
// The segment that CTA blockIdx.x began and others ended: its pieces' outputs by their totals, in order. 32
// dims of 128 pairs a CTA.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv8_prefill_combine_kernel(const __grid_constant__ PrefillArgs a) {
  using S = Shape<D, sizeof(T) == 4>;
  grid_dependency_wait();
  grid_launch_dependents();
  const int4 rec = a.record[blockIdx.x];
  if (rec.w < 2) return;
  const Work w = work_of<S>(a, rec.x);
  const int r = (int)(blockIdx.y / (D / 32)) * 128 + (int)threadIdx.x % 128, c0 = (int)(blockIdx.y % (D / 32)) * 8 + (int)threadIdx.x / 128 * 4;
  const long long pair = (long long)rec.y * S::PAIRS + r;
  if (pair >= w.pairs) return;
  auto slot = [&](int i) { return (size_t)(2 * ((int)blockIdx.x + i) + (i == 0)); };
  float top = -INFINITY;
  for (int i = 0; i < rec.w; ++i) {
    const float2 ml = a.part_ml[slot(i) * S::PAIRS + r];
    if (ml.y != 0.f) top = fmaxf(top, ml.x);
  }
  float all = 0.f;
  for (int i = 0; i < rec.w; ++i) {
    const float2 ml = a.part_ml[slot(i) * S::PAIRS + r];
    if (ml.y != 0.f) all += ml.y * exp2f(ml.x - top);
  }
  const float inv = all == 0.f ? 0.f : 1.f / all;
  float4 y[4] = {};
  for (int i = 0; i < rec.w; ++i) {
    const float2 ml = a.part_ml[slot(i) * S::PAIRS + r];
    if (ml.y == 0.f) continue;
    const float f = ml.y * exp2f(ml.x - top) * inv;  // (at most 1: no sum of large values leaves the range)
    const float4* o = a.part_o + (slot(i) * (D / 4) + c0) * S::PAIRS + r;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 x = o[(size_t)c * S::PAIRS];
      y[c].x = fmaf(x.x, f, y[c].x), y[c].y = fmaf(x.y, f, y[c].y), y[c].z = fmaf(x.z, f, y[c].z), y[c].w = fmaf(x.w, f, y[c].w);
    }
  }
  T* to = static_cast<T*>(a.out) + (long long)(w.r0 + pair / a.group) * a.ldo + ((size_t)rec.z * a.group + pair % a.group) * D + 4 * c0;
#pragma unroll
  for (int c = 0; c < 4; ++c) store4<T>(to + 4 * c, y[c]);
}

template <typename T, int D>
cudaError_t launch_shape(const PrefillArgs& a, cudaStream_t s) {
  using S = Shape<D, sizeof(T) == 4>;
  static int attr_set[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = cudaSuccess;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kv8_prefill_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv8_prefill_kernel<T, D>, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)a.ctas, S::MT * (D / 32));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv8_prefill_combine_kernel<T, D>, a);
}
template <typename T>
cudaError_t launch_typed(const PrefillArgs& a, cudaStream_t s) {
  return a.v.dim == 64 ? launch_shape<T, 64>(a, s) : (a.v.dim == 128 ? launch_shape<T, 128>(a, s) : launch_shape<T, 256>(a, s));
}

constexpr int pairs_of(int dim) { return dim <= 128 ? 256 : 128; }
// bytes of a piece's outputs, totals and maxima
size_t piece_bytes(int dim) { return (size_t)pairs_of(dim) * dim * 4; }

}  // namespace

size_t kv8_prefill_scratch(const Kv8View& v, int type, int) {
  const size_t ctas = num_sms();
  return ctas * (16 + 2 * (piece_bytes(v.dim) + pairs_of(v.dim) * 8)) + (type == APR_T_F32 ? ctas * piece_bytes(v.dim) : 0);
}

cudaError_t launch_kv8_prefill(const Kv8View& v, int type, const void* q, long long ldq, void* out, long long ldo,
                               int heads, float scale, void* scratch, cudaStream_t s) {
  const size_t ctas = num_sms();
  PrefillArgs a{v, q, out, ldq, ldo, heads, heads / v.kv_heads, scale * 1.4426950408889634f, (int)ctas};
  uint8_t* at = static_cast<uint8_t*>(scratch);
  a.part_o = reinterpret_cast<float4*>(at);
  at += 2 * ctas * piece_bytes(v.dim);
  a.part_ml = reinterpret_cast<float2*>(at);
  at += 2 * ctas * pairs_of(v.dim) * 8;
  a.record = reinterpret_cast<int4*>(at);
  a.mean = reinterpret_cast<float4*>(at + ctas * 16);
  if (type == APR_T_F32) return launch_typed<float>(a, s);
  if (type == APR_T_F16) return launch_typed<__half>(a, s);
  return launch_typed<__nv_bfloat16>(a, s);
}

}  // namespace apr
