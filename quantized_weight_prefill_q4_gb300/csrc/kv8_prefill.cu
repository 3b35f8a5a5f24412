// Attention of chunks of rows over their sequences' 8-bit paged KV caches
// (include/apr_kv8.h): for each (row, head) pair
//   p_j = softmax_j(scale q . (c_j s)),  out = sum_j p_j (c'_j s'),  j <= its position
//
// Bound. 4 D operations a pair and position, and every code is read once for 128 or 256
// pairs, so the tensor cores bound it: M = 128 pairs of one KV head a tile, keys in
// tiles of 128 or 64. Both products take fp16: codes are exact in it, a page's
// scale is a factor of 32 or more neighbouring scores (K) or weights (V).
//
// Segments. A segment is MT * 128 (row, head) pairs of a sequence that read one KV head,
// over all positions that its last row sees. What segments cost (positions, and a start
// worth START of them) is numbered through, a sequence's as a quadratic in closed form, and each CTA takes an
// equal, contiguous share: chunks of any lengths in one batch keep every SM equally busy. A
// segment within one share is finished there; of the others each CTA that has a piece
// writes its outputs, reference maximum and total, and a second kernel combines them in order.
//
// A CTA, one on each SM. The roles hand work to each other through mbarriers:
//   softmax    four warps for each M tile, a thread a pair (tensor memory lane): they
//              write q into shared memory, then per key tile read the scores, move the
//              running maximum and sum, and write the weights over the scores in tensor memory; O is
//              rescaled only when a maximum grows by more than 2^MOVE
//   one warp   looks up the pages and copies codes, a page's part of a tile at a time, into slots as they lie in memory
//   converters turn those into fp16 tiles in a ring of slots, rows of 128 bytes
//              swizzled for the tensor cores, dims contiguous: the product's k side for K, its N side for V
//              (loads straight from global memory held up every tile's fence until they landed: 2044 us, 1063 from the slots)
//   one warp   issues S = Q K^T (both from shared memory) and O += P V (P from tensor memory)
//   one warp   finds the next piece of the CTA's share
// With two M tiles (up to 128 dims) the tensor cores work on one while the other's softmax runs; with
// one on the next key tile's scores. Scores are issued into what the weights of the product ahead of them are read from (with two buffers,
// of the one before that), without a wait for its end. That rests on an SM's tensor pipe taking one CTA's products in the order of
// their issue, of whatever accumulator and shape; PTX promises it for products that share both. A weight read too late would
// be a score's bits, off by more than any tolerance of the tests, which hold for every head dim and type; and 1800 calls of 90 shapes gave
// the same bits with the wait. It would take 8 % of the time (2048 rows over 40011 positions 929 us, seven sequences of 900 to 9000 255),
// 1 to 4 % with two buffers.
//
// float32 rows: q and the weights enter as two fp16 pieces each (22 bits), twice the
// products. Of 16-bit rows the weights are one fp16 number: each is off by 2^-11 of itself at the most, fp16 outputs by 2.8e-4 of their
// norm in all, of which their own rounding is 2.0e-4; bf16 outputs by their rounding, 1.7e-3. With two pieces that would be 2.0e-4, in more
// than twice the time (2048 rows over 40011 positions 2004 us, 1024 over 8192 240, seven sequences of 900 to 9000 442).
//
// Weights. A pair's weights are 2^11 p v, p against a reference at most MOVE (base 2) below the
// maximum, v the page's V scale over a power of two R that no scale so far exceeds, a quarter or more for the largest: at most 2^15, and
// 2^9 or more for the largest one. fp16's steps end at 2^-24, so that a weight is kept to 2^-34 of the largest (times the largest
// scale over its own); 2^7 and a MOVE of 8 kept 2^-30. O is rescaled a little more often (2048 rows over 40011 positions 856 us, 853 with
// 8; seven sequences of 900 to 9000 242 and 238).
//
// Measured (calls in a graph; bf16 products of a library run at 1928 TFLOP/s in a burst, 1745 sustained):
//   2048 rows over 40011 positions, 32 heads over 8 of 128, bf16   856 us, 1529 TFLOP/s
//   8192 over 131072, 32 over 8 of 128, bf16                       11.5 ms, 1482
//   1024 over 8192, 32 over 8 of 128, bf16                         117 us, 1100 (starts, ends and the combination: 27)
//   1024 over 8192, 16 over 4 of 256, bf16                         136 us, 947 (one M tile: a tile's scores wait for its softmax's end)
//   1024 over 8192, 32 over 8 of 64, fp16                          92 us, 700 (54 of it exponentials, 16 a cycle and SM)
//   1024 over 8192, 32 over 8 of 128, float32                      262 us, 491, twice as many products done
//   512 over 512, 32 over 8 of 128, bf16                           26 us
//   37 over 731, 8 over 2 of 64, fp16                              17 us (two launches, each role's first instructions, a tile's way through the roles)
//   64 sequences' next tokens (300 to 18700 positions, 32 heads over 8 of 128, bf16) beside 1024 rows over 8192: 382 us, where 117 and, by
//   kv8_attention.cu, 102 would do one after the other: a segment of few rows takes as long as one of 256

#include "apr_internal.h"
#include "host_common.h"
#include "kv8.cuh"

namespace apr {
namespace {

// Positions that a segment's start and end are worth (2048 rows over 2048, 32 heads over 8 of 128: 73 us; when it was chosen 68, 82 with
// 256, 108 with 128, 69 with 1024). Whatever its rows: see the last line above.
constexpr int START = 512;
constexpr int MIN_TILES = 2;     // of a CTA's share
// Shares that the costliest segment is long, about, at the most: as shares begin anywhere in it, it is cut into one or two pieces more. More
// pieces take longer to combine than they save (64 rows over 20000, 8 heads over 2 of 64: 40 us; when it was chosen 36, 39 with 32, 75 in
// the 76 pieces that every SM would have one of; 32 rows over 100000 89 us, 119 with 12).
constexpr int MOST_PIECES = 24;
constexpr float MOVE = 4.f;
// A wait for the next piece, or for the last one to be over, lasts as long as a piece: 2^30 positions take
// some 40 s. (Every wait within one is short, and one that runs out ends these, too.)
constexpr unsigned long long PIECE_LIMIT_NS = 300000000000ull;
constexpr int MMA_WARP = 12, PIECE_WARP = 13, COPY_WARP = 14, THREADS = 512;  // (the last warp has nothing to do)

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
  float4* mean;      // [ctas][D / 4][pairs] the mean taken over
  float2* mean_ml;   // [ctas][pairs] its reference and total
};

template <int D_, bool TWO_>
struct Shape {
  static constexpr int D = D_;
  static constexpr bool TWO = TWO_;                        // two fp16 pieces of q and of the weights
  static constexpr int MT = D <= 128 ? 2 : 1;              // M tiles
  static constexpr int PAIRS = 128 * MT;
  static constexpr int KT = MT == 2 && !TWO ? 128 : 64;    // keys of a tile
  static constexpr int NB = KT == 128 ? 1 : 2;             // buffers of scores of an M tile
  static constexpr int GROUPS = KT / 32;                   // of 32 positions, within one page each
  static constexpr int PIECES = TWO ? 2 : 1;
  static constexpr int PANEL = KT * 128;                   // bytes of 64 dims of a tile
  static constexpr int SLOT = KT * D * 2;
  static constexpr int Q_BYTES = MT * PIECES * 128 * D * 2;
  // fp16 slots and slots of codes as they lie in memory
  static constexpr int RAW = KT * D;
  static constexpr int LEFT = 226 * 1024 - Q_BYTES;
  static constexpr int SLOTS = LEFT >= 4 * (SLOT + RAW) ? (LEFT / (SLOT + RAW) < 6 ? LEFT / (SLOT + RAW) : 6) : (LEFT >= 3 * (SLOT + RAW) ? 3 : 2);
  static constexpr int RAWS_FIT = (LEFT - SLOTS * SLOT) / RAW;
  static constexpr int RAWS = RAWS_FIT < 6 ? RAWS_FIT : 6;
  static constexpr int SMEM = Q_BYTES + SLOTS * SLOT + RAWS * RAW + 1024;
  static constexpr int SOFT = 4 * MT, CONV = MMA_WARP - SOFT;  // warps
  // registers a thread of each role; as launched: 128
  static constexpr int SOFT_REGS = MT == 2 ? 192 : 208, CONV_REGS = MT == 2 ? 64 : 88, MMA_REGS = MT == 2 ? 64 : 128;
  static_assert(32 * (SOFT * SOFT_REGS + CONV * CONV_REGS + 4 * MMA_REGS) <= THREADS * 128, "registers");
  // converter warps of a chunk: with eight two teams, every other chunk each (256 dims 154 -> 127 us; two teams of two warps took
  // longer than one of four, 956 us instead of 851)
  static constexpr int TEAMS = CONV / 4, TEAM = 4;
  static constexpr int EACH = KT * D / 16 / (32 * TEAM);   // 16-byte pieces of a chunk that a converter thread has
  // tensor memory columns: O of each M tile, then its buffers of scores, which the weights take over
  static constexpr int COL_S = MT * D;
  static_assert(COL_S + NB * MT * KT <= 512 && PIECES * KT / 2 <= KT, "tensor memory");
  static_assert(SLOTS >= 2 && RAWS >= 2 && SMEM + 1024 <= 232448, "shared memory");
  static_assert(EACH >= 1 && KT * D / 16 % (32 * TEAM) == 0, "converters");
  // Positions after which O is taken over into a float32 mean: its sums lose some 2e-8 of themselves at each step of 16
  // positions, always towards zero. 6e-7 in 512 for float32 rows, within a piece; 8e-5 in 65536 for 16-bit rows, whose weights and outputs
  // are rounded by 2e-4 or more, where a piece is cut (code for it in the loop over key tiles took 20% longer for all). Both are in the header.
  static constexpr int FOLD_TILES = (TWO ? 512 : 65536) / KT;
};

// ---------------------------------------------------------------- the work
// a / b of numbers that are not negative, in 32 bits where they are that small (a division of 64 takes hundreds of cycles).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
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
  const int sees = w.first + (int)quotient(last, a.group) + 1;
  return max(1, (sees + S::KT - 1) / S::KT);
}
// The key tile of a segment that a share begins with which begins `at` into the segment's cost.
template <class S>
__device__ __forceinline__ int tile_at(const PrefillArgs& a, long long at, int tiles) {
  const long long in = at - (long long)START * a.group, step = (long long)S::KT * a.group;
  return in <= 0 ? 0 : (int)min((long long)tiles, quotient(in + step - 1, step));
}
// A piece, as the roles see it: key tiles k0 .. k1 - 1 of the `tiles` of a segment (k1 == 0: no more pieces).
struct Piece {
  int b, g;          // sequence and KV head
  int len, first, r0;
  int k0, k1, tiles;
  int from, to;      // the CTA's part of the segment, of which this may be one of several cuts
  int np;            // pairs of the segment, from p0 of the sequence's on
  long long p0;
};

// The pieces of a CTA's share, one after the other; a whole warp calls it.
template <class S>
struct Pieces {
  int b;
  long long u, end, seq_u0, share, total;  // CTA c's share: share * c .. share * (c + 1) - 1, within the total

  // The next piece, and of how many pieces its segment is made where the piece begins it.
  __device__ __forceinline__ bool next(const PrefillArgs& a, Piece& p, int& t, int& made_of) {
    const int lane = threadIdx.x & 31;
    while (u < end && b < a.v.num_seqs) {
      const Work w = work_of<S>(a, b);
      const long long all = cost_all<S>(a, w);
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
      int lo = 0, hi = w.segments;  // the last segment that begins at or before it
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (a.v.kv_heads * cost_before<S>(w, mid) <= at)
          lo = mid;
        else
          hi = mid;
      }
      const long long before = a.v.kv_heads * cost_before<S>(w, lo), one = cost<S>(w, lo);
      t = lo;
      p.b = b;
      p.g = (int)min(quotient(at - before, one), (long long)a.v.kv_heads - 1);
      const long long seg_u0 = seq_u0 + before + p.g * one, seg_end = seg_u0 + one;
      p.tiles = key_tiles<S>(a, w, lo);
      p.k0 = u == seg_u0 ? 0 : tile_at<S>(a, u - seg_u0, p.tiles);
      p.k1 = end >= seg_end ? p.tiles : tile_at<S>(a, end - seg_u0, p.tiles);
      u = min(end, seg_end);
      if (p.k0 >= p.k1) continue;
      p.len = w.len, p.first = w.first, p.r0 = w.r0;
      p.p0 = (long long)lo * S::PAIRS;
      p.np = (int)min((long long)S::PAIRS, w.pairs - p.p0);
      p.from = p.k0, p.to = p.k1;
      made_of = 1;
      if (p.k0 == 0 && p.k1 < p.tiles)
        for (long long x = end; x < min(seg_end, total) && tile_at<S>(a, x - seg_u0, p.tiles) < p.tiles; x += share) ++made_of;
      return true;
    }
    return false;
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
  if (group * 32ll >= p.len) return 0;
  const int pos = group * 32, page = max(kv8_page(a.v, p.b, pos >> a.v.page_shift), 0);
  return (uint32_t)(kv8_scale_at(a.v, page, p.g) << (a.v.page_shift - 5)) +
         (uint32_t)((pos >> 5) & ((1 << (a.v.page_shift - 5)) - 1));
}
// The scales of a group of 32 positions.
struct GroupScales {
  float k, v;
};
__device__ __forceinline__ GroupScales group_scales(const PrefillArgs& a, const Piece& p, int group) {
  if (group * 32ll >= p.len) return GroupScales{0.f, 0.f};
  const size_t at = kv8_scale_at(a.v, max(kv8_page(a.v, p.b, group * 32 >> a.v.page_shift), 0), p.g);
  return GroupScales{a.v.k_scale[at], a.v.v_scale[at]};
}

// ---------------------------------------------------------------- tensor core operands
// D[tmem] (+)= A . B, both from shared memory. As for mma_f16_ts_elect, the warp stays together and what the
// instruction takes is the same for all of it, known to be so from a shuffle: in uniform registers, where
// a product takes them from (from others each took 100 cycles to issue).
__device__ __forceinline__ void mma_f16_ss_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
// A shared memory descriptor but for its start address: rows of 128 bytes, swizzled, groups of 8 of them 1024
// bytes apart (stride byte offset), the next 64 columns `panel` bytes on (leading byte offset: counts where N is contiguous, as
// in V as the second product's B).
constexpr uint64_t operand_desc(uint32_t panel) {
  return (uint64_t)(panel >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
constexpr uint32_t N_MAJOR_B = 1u << 16;

// Registers of a warpgroup's threads from here on (a rise waits for those that others give up).
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

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
// The exponent of a row's largest magnitude (kept to 2^+-120: beyond, the row enters scaled less, its products still in range).
__device__ __forceinline__ int q_exponent(float top) {
  return top <= FLT_MAX ? min(max((int)(__float_as_uint(top) >> 23) - 127, -120), 120) : 0;
}
// The elements of 16 bytes of a row.
template <typename T, int N>
__device__ __forceinline__ void values_of(const uint4& w, float (&x)[N]) {
  if constexpr (N == 4)
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  else
    values8(Vec8<T>{w}, x);
}
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
  uint8_t* raw = ring + S::SLOTS * S::SLOT;
  __shared__ uint64_t raw_full[S::RAWS], raw_empty[S::RAWS], full[S::SLOTS], empty[S::SLOTS], q_full[2], s_full[4], p_full[4], o_done[2], o_last[2], piece_full[2],
      piece_empty[2], drain;
  __shared__ Piece s_piece[2];
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_words[2];  // the second is never set: the drain's wait ignores the abort
  __shared__ long long s_scan[THREADS / 32], s_largest[THREADS / 32], s_found[1];
  __shared__ int s_found_b;
  volatile int* abort_flag = abort_words;
  const Kv8View& v = a.v;
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);

  // ---- what the sequences cost, and where this CTA's share begins: a thread counts `run` neighbouring sequences
  const int run = (v.num_seqs + THREADS - 1) / THREADS;
  const int my_b0 = min((int)threadIdx.x * run, v.num_seqs), my_b1 = min(my_b0 + run, v.num_seqs);
  long long mine = 0, largest = 0;  // what they cost, and the most that a segment of theirs does
  for (int b = my_b0; b < my_b1; ++b) {
    const Work w = work_of<S>(a, b);
    mine += cost_all<S>(a, w);
    if (w.segments > 0) largest = max(largest, cost<S>(w, w.segments - 1));
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
    largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, o));
  }
  if (lane == 31) s_scan[warp] = inc, s_largest[warp] = largest;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::SLOTS; ++i) {
      mbar_init(&full[i], S::TEAM);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < S::RAWS; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], S::TEAM);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[2 * i], 1);
      mbar_init(&s_full[2 * i + 1], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_last[i], 1);
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], MMA_WARP + 2);
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
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) my_u0 += s_scan[w];
    total += s_scan[w];
    largest = max(largest, s_largest[w]);
  }
  const long long share = max(quotient(max(total, 0ll) + a.ctas - 1, a.ctas), max((long long)MIN_TILES * S::KT * a.group, quotient(largest, MOST_PIECES)));
  const long long u = share * blockIdx.x, u_end = min(u + share, total);
  const bool idle = u >= total;
  if (!idle && my_u0 <= u && u < my_u0 + mine) {
    int b = my_b0;
    long long at = my_u0;
    for (long long n; b + 1 < my_b1 && at + (n = cost_all<S>(a, work_of<S>(a, b))) <= u; ++b) at += n;
    s_found_b = b;
    s_found[0] = at;
  }
  __syncthreads();
  int ok = 1;
  auto wait = [&](uint64_t* bar, int phase) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(phase & 1), abort_flag, v.status));
    return ok;
  };
  auto wait_piece = [&](uint64_t* bar, int phase) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait_for(bar, (uint32_t)(phase & 1), abort_flag, v.status, PIECE_LIMIT_NS));
    return ok;
  };
  // the i-th piece, once it is known; and no longer looked at
  auto piece_is = [&](int i) { return wait_piece(&piece_full[i & 1], i >> 1) && s_piece[i & 1].k1 > 0; };
  auto piece_done = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[i & 1]);
  };

  if (warp < S::SOFT) {
    // ------------------------------------------------ softmax
    more_registers<S::SOFT_REGS>();
    const int m = warp / 4, r = (int)threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16), o_col = lanes + m * D;
    const T* q = static_cast<const T*>(a.q);
    T* out = static_cast<T*>(a.out);
    int cnt = 0, mine_so_far = 0;  // key tiles, and pieces with pairs of this M tile, so far
    for (int ip = 0; piece_is(ip); piece_done(ip), ++ip) {
      const Piece& p = s_piece[ip & 1];
      if (128 * m >= p.np) continue;
      auto scales_of = [&](int group) { return group_scales(a, p, group); };
      Window<GroupScales, decltype(scales_of)> scales;
      scales.begin(p.k0 * S::GROUPS, scales_of);
      // (what of a row the key tiles do not need is found again where it is)
      const auto row_of = [&](bool& live) {
        live = 128 * m + r < p.np;
        return (int)quotient(p.p0 + 128 * m + (live ? r : 0), a.group);
      };
      const auto at_of_row = [&](int i, long long ld) {
        const long long pair = p.p0 + 128 * m + (128 * m + r < p.np ? r : 0);
        return (long long)(p.r0 + i) * ld + ((long long)p.g * a.group + pair - (long long)i * a.group) * D;
      };
      bool live;
      const int i = row_of(live);
      // ---- the warp's 32 rows, some lanes a row: fp16 pieces times a power of two that brings a row's largest
      // magnitude into [1, 2); a row with a NaN or an infinity as zeros, its scores' factor NaN
      const long long q_at = at_of_row(i, a.ldq);
      float top = 0.f;  // of this thread's row
      {
        constexpr int N = 16 / sizeof(T), VECS = D / N, LR = VECS < 32 ? VECS : 32, V = VECS / LR;  // elements of 16 bytes; a row's lanes, and what a lane has of it
        constexpr int RS = 32 / LR, BATCH = 8;
        const int in_row = lane % LR;
        const unsigned alive = __ballot_sync(0xffffffffu, live);
        uint8_t* rows = sQ + m * S::PIECES * 128 * D * 2;
#pragma unroll 1
        for (int b0 = 0; b0 < 32 / RS; b0 += BATCH) {
          uint4 x[BATCH][V];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const int owner = (b0 + k) * RS + lane / LR;
            const T* from = q + __shfl_sync(0xffffffffu, q_at, owner & 31);
#pragma unroll
            for (int e = 0; e < V; ++e)
              if (owner < 32) x[k][e] = *reinterpret_cast<const uint4*>(from + (e * LR + in_row) * N);
          }
          float most[BATCH];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            most[k] = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
              float y[N];
              values_of<T>(x[k][e], y);
#pragma unroll
              for (int h = 0; h < N; ++h) most[k] = fmaxf(most[k], y[h] == y[h] ? fabsf(y[h]) : INFINITY);
            }
          }
#pragma unroll
          for (int o = LR / 2; o > 0; o >>= 1)  // (the rows' steps side by side: a shuffle takes 25 cycles)
#pragma unroll
            for (int k = 0; k < BATCH; ++k) most[k] = fmaxf(most[k], __shfl_xor_sync(0xffffffffu, most[k], o));
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const float mine = __shfl_sync(0xffffffffu, most[k], (lane - (b0 + k) * RS) * LR & 31);
            if (lane / RS == b0 + k) top = mine;
          }
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const int owner = (b0 + k) * RS + lane / LR, R = warp % 4 * 32 + owner;
            if (owner >= 32) break;
            const bool zero = !(most[k] <= FLT_MAX) || !(alive >> owner & 1);
            const float down = zero ? 0.f : __uint_as_float((uint32_t)(127 - q_exponent(most[k])) << 23);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              float y[N];
              values_of<T>(x[k][e], y);
              uint32_t hi[N / 2], lo[N / 2];
#pragma unroll
              for (int h = 0; h < N / 2; ++h) {
                const float y0 = zero ? 0.f : y[2 * h] * down, y1 = zero ? 0.f : y[2 * h + 1] * down;
                hi[h] = half2_bits(y0, y1);
                const float2 f = half2_values(hi[h]);
                lo[h] = half2_bits(y0 - f.x, y1 - f.y);
              }
              const int d = (e * LR + in_row) * N;
              uint8_t* to = rows + (d / 64) * 128 * 128 + R * 128 + (((d / 8 % 8) ^ (R & 7)) << 4) + d % 8 * 2;
              if constexpr (N == 8) {
                *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              } else {
                *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(to + 128 * D * 2) = make_uint2(lo[0], lo[1]);
              }
            }
          }
        }
      }
      const int sees = live ? min(p.len, p.first + i + 1) : 0;  // positions
      // (of a row that sees none, as in a slot without a sequence, whatever it holds: its outputs are zeros)
      const float factor = !(top <= FLT_MAX) && sees > 0 ? __int_as_float(0x7fffffff)
                                                         : a.scale_log2 * __uint_as_float((uint32_t)(127 + q_exponent(top)) << 23);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[m]);
      ++mine_so_far;

      float ref = -INFINITY, run_max = -INFINITY, sum = 0.f;
      float R = 0x1p-100f;  // a power of two
      float mean_ref = -INFINITY, mean_sum = 0.f;  // of the mean taken over
      const int k0 = p.k0, k1 = p.k1;
      // ---- O, with the mean taken over so far, to the mean, a piece's outputs or the rows
      // (co, cm: what O and the mean count for)
      float co, cm;
      auto join = [&] {
        // (a side without weights has no say: a row that sees nothing of a cut has a reference of 0 there, however low its scores were)
        const float top_ref = sum == 0.f ? mean_ref : (mean_sum == 0.f ? ref : fmaxf(ref, mean_ref));
        const float wn = sum == 0.f ? 0.f : exp2f(ref - top_ref), wm = mean_sum == 0.f ? 0.f : exp2f(mean_ref - top_ref);
        const float all = sum * wn + mean_sum * wm, inv = all == 0.f ? 0.f : 1.f / all;
        co = R * 0x1p-11f * (wn * inv), cm = wm * mean_sum * inv;
        const bool more = mean_sum != 0.f;
        mean_ref = top_ref;
        mean_sum = all;
        sum = 0.f;
        return more;
      };
      // O into the mean, 64 dims of which are on their way together (128 no longer fit the registers; 32 for 16-bit rows)
      auto fold = [&] {
        constexpr int G = S::TWO ? 2 : 1;
        const bool more = join();
        float4* mean = a.mean + (size_t)blockIdx.x * (D / 4) * S::PAIRS + 128 * m + r;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 32; c0 += G, mean += (size_t)8 * G * S::PAIRS) {
          float4 x[G][8];
          if (S::TWO && more) {
#pragma unroll
            for (int k = 0; k < 8 * G; ++k) x[k / 8][k % 8] = mean[(size_t)k * S::PAIRS];
          }
#pragma unroll
          for (int cc = 0; cc < G; ++cc) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(o_col + 32 * (c0 + cc), o);
            tmem_ld_wait_regs(o);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float4 y = make_float4(__uint_as_float(o[4 * k]) * co, __uint_as_float(o[4 * k + 1]) * co,
                                     __uint_as_float(o[4 * k + 2]) * co, __uint_as_float(o[4 * k + 3]) * co);
              if (more) {
                const float4 z = S::TWO ? x[cc][k] : mean[(size_t)(8 * cc + k) * S::PAIRS];
                y.x = fmaf(z.x, cm, y.x), y.y = fmaf(z.y, cm, y.y), y.z = fmaf(z.z, cm, y.z), y.w = fmaf(z.w, cm, y.w);
              }
              if (mean_sum == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);  // (whatever O held)
              mean[(size_t)(8 * cc + k) * S::PAIRS] = y;
            }
          }
        }
      };
      // O and the mean to a piece's outputs or the rows
      auto finish = [&] {
        const bool partial = p.to - p.from < p.tiles;
        const int slot = 2 * (int)blockIdx.x + (p.from == 0);
        const bool more = join();
        float4* mean = a.mean + (size_t)blockIdx.x * (D / 4) * S::PAIRS + 128 * m + r;
        float4* part = a.part_o + (size_t)slot * (D / 4) * S::PAIRS + 128 * m + r;
        bool live;
        const long long out_at = at_of_row(row_of(live), a.ldo);
        // the rows that this lane's 16 bytes go to: 4 it + lane / 8
        long long to[8];
        const unsigned alive = __ballot_sync(0xffffffffu, live);
        if (!partial) {
#pragma unroll
          for (int it = 0; it < 8; ++it)
            to[it] = __shfl_sync(0xffffffffu, out_at, it * 4 + lane / 8) + (lane & 7) * (16 / (int)sizeof(T));
        }
        // (rows of T leave through the warp's own rows of q's place, which no product reads any more: 128 bytes of
        // a row together instead of 16)
        constexpr int DIMS = 128 / sizeof(T);
        float4 x[2][8];  // the mean so far, 32 dims ahead (16-bit rows: when it is added, which seldom is)
        if (S::TWO && more) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[0][k] = mean[(size_t)k * S::PAIRS];
        }
#pragma unroll 1
        for (int c0 = 0; c0 < D / 32; c0 += 2) {
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int c = c0 + cc;
            uint32_t o[32];
            tmem_ld_32x32b_x32(o_col + 32 * c, o);
            if (S::TWO && more && c + 1 < D / 32) {
#pragma unroll
              for (int k = 0; k < 8; ++k) x[1 - cc][k] = mean[(size_t)(8 * c + 8 + k) * S::PAIRS];
            }
            tmem_ld_wait_regs(o);
            uint8_t* row = sQ + m * S::PIECES * 128 * D * 2 + 32 * c / DIMS * (128 * 128) + r * 128;
            uint2 half_chunk = make_uint2(0, 0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float4 y = make_float4(__uint_as_float(o[4 * k]) * co, __uint_as_float(o[4 * k + 1]) * co,
                                     __uint_as_float(o[4 * k + 2]) * co, __uint_as_float(o[4 * k + 3]) * co);
              if (more) {
                const float4 z = S::TWO ? x[cc][k] : mean[(size_t)(8 * c + k) * S::PAIRS];
                y.x = fmaf(z.x, cm, y.x), y.y = fmaf(z.y, cm, y.y), y.z = fmaf(z.z, cm, y.z), y.w = fmaf(z.w, cm, y.w);
              }
              if (mean_sum == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);  // (whatever O held)
              if (partial) {
                part[(size_t)(8 * c + k) * S::PAIRS] = y;
              } else if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(row + ((k ^ (r & 7)) << 4)) = y;
              } else {
                const uint2 h = make_uint2(pack2<T>(y.x, y.y), pack2<T>(y.z, y.w));
                if (k & 1)
                  *reinterpret_cast<uint4*>(row + (((32 * c % DIMS / 8 + k / 2) ^ (r & 7)) << 4)) =
                      make_uint4(half_chunk.x, half_chunk.y, h.x, h.y);
                else
                  half_chunk = h;
              }
            }
          }
          if (!partial) {
            __syncwarp();
#pragma unroll
            for (int b = 0; b < 64 / DIMS; ++b) {  // 128-byte blocks of the 64 dims
              const int block = 32 * c0 / DIMS + b;
#pragma unroll
              for (int it = 0; it < 8; ++it) {
                const int rr = it * 4 + lane / 8, R = warp % 4 * 32 + rr;
                const uint4 y = *reinterpret_cast<const uint4*>(sQ + m * S::PIECES * 128 * D * 2 + block * (128 * 128) + R * 128 +
                                                                (((lane & 7) ^ (R & 7)) << 4));
                if (alive >> rr & 1) *reinterpret_cast<uint4*>(out + to[it] + block * DIMS) = y;
              }
            }
          }
        }
      };
      bool fresh = true;  // O holds nothing yet
#pragma unroll 1
      for (int j = k0; j < k1; ++j, ++cnt) {
        const int buf = S::NB == 2 ? 2 * m + (cnt & 1) : m, phase = S::NB == 2 ? cnt >> 1 : cnt;
        scales.reach(j * S::GROUPS, scales_of);
        float ks[S::GROUPS], vs[S::GROUPS];
        float vmax = 0.f;
#pragma unroll
        for (int c = 0; c < S::GROUPS; ++c) {
          ks[c] = __shfl_sync(0xffffffffu, scales.now.k, j * S::GROUPS + c - scales.base) * factor;
          ks[c] = ks[c] == 0.f ? FLT_MIN : ks[c];  // (as good as 0 for a score, but minus infinity stays that)
          vs[c] = __shfl_sync(0xffffffffu, scales.now.v, j * S::GROUPS + c - scales.base);
          vmax = fmaxf(vmax, vs[c]);
        }
        // (these scores' completion covers every product issued before them: with one buffer the last tile's O, with two the
        // one before that, so that a wait for the last one, by parity, cannot be a phase behind)
        if (!wait(&s_full[buf], phase)) break;
        tc_fence_after();
        if (S::TWO && j > k0 && (j - k0) % S::FOLD_TILES == 0) {
          if (S::NB == 2 && !wait(&o_done[m], cnt - 1)) break;
          tc_fence_after();
          fold();
          fresh = true;
        }
        const uint32_t s_col = lanes + S::COL_S + buf * S::KT;
        uint32_t s[S::KT];
#pragma unroll
        for (int c = 0; c < S::GROUPS; ++c) tmem_ld_32x32b_x32(s_col + 32 * c, s + 32 * c);
        tmem_ld_wait_regs(s);
#pragma unroll
        for (int c = 1; c < S::GROUPS; ++c) regs_after_wait(s + 32 * c);
        const int left = sees - j * S::KT;  // positions of the tile that the row sees
        if (!__all_sync(0xffffffffu, left >= S::KT)) {
#pragma unroll
          for (int k = 0; k < S::KT; ++k) s[k] = k < left ? s[k] : 0xff800000u;
        }
        float tile_max = -INFINITY;
#pragma unroll
        for (int c = 0; c < S::GROUPS; ++c) {
          float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            x[0] = fmaxf(fmaxf(x[0], __uint_as_float(s[32 * c + k])), __uint_as_float(s[32 * c + k + 1]));
            x[1] = fmaxf(fmaxf(x[1], __uint_as_float(s[32 * c + k + 2])), __uint_as_float(s[32 * c + k + 3]));
          }
          tile_max = fmaxf(tile_max, fmaxf(x[0], x[1]) * ks[c]);
        }
        run_max = fmaxf(run_max, tile_max);
        // ---- the reference, and R: O moves with them
        const bool grow = vmax > R;
        if (fresh) {
          ref = run_max == -INFINITY ? 0.f : run_max;
          if (grow) {
            R = __uint_as_float(min((__float_as_uint(vmax) & 0x7f800000u) + (2u << 23), 0x7e800000u));
          }
        } else if (grow || __any_sync(0xffffffffu, run_max > ref + MOVE)) {
          if (S::NB == 2 && !wait(&o_done[m], cnt - 1)) break;
          tc_fence_after();
          const float new_ref = run_max > ref ? run_max : ref;
          float f = exp2f(ref - new_ref);
          sum *= f;
          ref = new_ref;
          if (grow) {
            const float new_R = __uint_as_float(min((__float_as_uint(vmax) & 0x7f800000u) + (2u << 23), 0x7e800000u));
            f *= R * (1.f / new_R);
            R = new_R;
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
#pragma unroll
        for (int c = 0; c < S::GROUPS; ++c) {
          const float w = vs[c] * __uint_as_float((265u << 23) - __float_as_uint(R));  // * 2^11 / R
          const float2 k2 = make_float2(ks[c], ks[c]), r2 = make_float2(-ref, -ref), w2 = make_float2(w, w);
          float2 l = make_float2(0.f, 0.f);
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 y = make_float2(__uint_as_float(s[32 * c + 2 * k]), __uint_as_float(s[32 * c + 2 * k + 1]));
            float2 x = __ffma2_rn(y, k2, r2);
            x.x = exp2_fast(x.x), x.y = exp2_fast(x.y);
            l = __fadd2_rn(l, x);
            x = __fmul2_rn(x, w2);
            hi[k] = half2_bits(x.x, x.y);
            if constexpr (S::TWO) {
              const float2 f = half2_values(hi[k]);
              lo[k] = half2_bits(x.x - f.x, x.y - f.y);
            }
          }
          sum += l.x + l.y;
          tmem_st_32x32b_x16(s_col + 16 * c, hi);
          if constexpr (S::TWO) tmem_st_32x32b_x16(s_col + S::KT / 2 + 16 * c, lo);
        }
        tmem_st_wait();
        fresh = false;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      if (!ok || !wait(&o_last[m], mine_so_far - 1)) break;
      tc_fence_after();
      float2* mean_ml = a.mean_ml + (size_t)blockIdx.x * S::PAIRS + 128 * m + r;
      if (!S::TWO && p.k0 > p.from) {
        const float2 ml = *mean_ml;
        mean_ref = ml.x, mean_sum = ml.y;
      }
      if (!S::TWO && p.k1 < p.to) {
        fold();
        *mean_ml = make_float2(mean_ref, mean_sum);
      } else {
        finish();
        if (p.to - p.from < p.tiles)
          a.part_ml[(size_t)(2 * (int)blockIdx.x + (p.from == 0)) * S::PAIRS + 128 * m + r] = make_float2(mean_ref, mean_sum);
      }
      tc_fence_before();
    }
  } else if (warp < MMA_WARP) {
    // ------------------------------------------------ converters: chunks of K and V in the order in which they are used
    fewer_registers<S::CONV_REGS>();
    const int tid = ((int)threadIdx.x - 32 * S::SOFT) % (32 * S::TEAM), team = (warp - S::SOFT) / S::TEAM;
    constexpr int ROW = D / 16;                       // 16-byte pieces of a position's codes
    constexpr int STEP = 32 * S::TEAM / ROW;          // positions from one of a thread's pieces to the next
    const int key0 = tid / ROW, piece = tid % ROW, panel = piece / 4;
    uint32_t rs = team, slot_of = team, raw_phase = 0, phase = 1;  // of this team's next chunk
    for (int ip = 0; piece_is(ip); piece_done(ip), ++ip) {
      const int mine = 2 / S::TEAMS * (s_piece[ip & 1].k1 - s_piece[ip & 1].k0);
#pragma unroll 1
      for (int c = 0; c < mine; ++c) {
        if (!wait(&raw_full[rs], raw_phase) || !wait(&empty[slot_of], phase)) break;
        const uint8_t* from = raw + rs * S::RAW + tid * 16;
        uint8_t* slot = ring + slot_of * S::SLOT + panel * S::PANEL;
        constexpr int AHEAD = S::EACH < 8 ? S::EACH : 8;
#pragma unroll
        for (int i0 = 0; i0 < S::EACH; i0 += AHEAD) {
          uint4 x[AHEAD];
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) x[i] = *reinterpret_cast<const uint4*>(from + (i0 + i) * (32 * S::TEAM * 16));
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) {
            const int key = key0 + (i0 + i) * STEP;
            const uint32_t b[4] = {x[i].x ^ 0x80808080u, x[i].y ^ 0x80808080u, x[i].z ^ 0x80808080u, x[i].w ^ 0x80808080u};
            const uint4 y0 = make_uint4(half2_of_codes(b[0], 0x4140), half2_of_codes(b[0], 0x4342),
                                        half2_of_codes(b[1], 0x4140), half2_of_codes(b[1], 0x4342));
            const uint4 y1 = make_uint4(half2_of_codes(b[2], 0x4140), half2_of_codes(b[2], 0x4342),
                                        half2_of_codes(b[3], 0x4140), half2_of_codes(b[3], 0x4342));
            uint8_t* row = slot + key * 128;
            const int c8 = 2 * (piece & 3), odd = panel & 1;  // (neighbouring panels' stores go to different banks)
            *reinterpret_cast<uint4*>(row + (((c8 + odd) ^ (key & 7)) << 4)) = odd ? y1 : y0;
            *reinterpret_cast<uint4*>(row + (((c8 + 1 - odd) ^ (key & 7)) << 4)) = odd ? y0 : y1;
          }
        }
        fence_proxy_async_smem();  // (no load from global memory is on its way, which it would wait for)
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[rs]);
          mbar_arrive(&full[slot_of]);
        }
        for (int i = 0; i < S::TEAMS; ++i) {
          if (++rs == S::RAWS) rs = 0, raw_phase ^= 1;
          if (++slot_of == S::SLOTS) slot_of = 0, phase ^= 1;
        }
      }
      if (!ok) break;
    }
  } else {
    fewer_registers<S::MMA_REGS>();
  }
  if (warp == MMA_WARP) {
    // ------------------------------------------------ the products
    constexpr uint32_t IDESC_S = idesc_f16_f32(128, S::KT), IDESC_O = idesc_f16_f32(128, D) | N_MAJOR_B;
    const uint32_t base = uniform(tmem), q_at = uniform(smem_u32(sQ)) >> 4, ring_at = uniform(smem_u32(ring)) >> 4;
    constexpr uint64_t desc = operand_desc(16), v_desc = operand_desc(S::PANEL);
    uint32_t cnt0 = 0, cnt1 = 0, mine0 = 0, mine1 = 0;  // key tiles and pieces of each M tile, so far
    uint32_t k_slot = 0, k_phase = 0;                    // of the K chunk that is next
    for (int ip = 0; piece_is(ip); piece_done(ip), ++ip) {
      const uint32_t n = uniform(s_piece[ip & 1].k1 - s_piece[ip & 1].k0);
      const uint32_t nm = S::MT == 2 ? uniform(s_piece[ip & 1].np > 128 ? 2 : 1) : 1;
      uint32_t v_slot = 0, v_phase = 0;  // the slot, and its phase, of the V chunk that is next
      auto advance = [&](uint32_t& slot, uint32_t& phase) {
        if (++slot == S::SLOTS) slot = 0, phase ^= 1;
      };
      auto issue_s = [&](uint32_t x, uint32_t m) {
        const uint32_t buf = S::NB == 2 ? 2 * m + (x & 1) : m;
        if (m == 0 && !wait(&full[k_slot], k_phase)) return;
        tc_fence_after();
        const uint64_t kd = desc + (ring_at + k_slot * (S::SLOT >> 4));
#pragma unroll
        for (int s = S::PIECES - 1; s >= 0; --s) {  // the small piece first
          const uint64_t qd = desc + (q_at + (m * S::PIECES + s) * (128 * D * 2 >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_f16_ss_elect(base + S::COL_S + buf * S::KT, qd + (uint64_t)((kk / 4 * 128 * 128) >> 4) + 2 * (kk % 4),
                             kd + (uint64_t)((kk / 4 * S::PANEL) >> 4) + 2 * (kk % 4), IDESC_S, s != S::PIECES - 1 || kk != 0);
        }
        mma_commit_elect(&s_full[buf]);
        if (m == nm - 1) mma_commit_elect(&empty[k_slot]);
      };
      auto issue_o = [&](uint32_t x, uint32_t m, bool fresh, bool last) {
        const uint32_t buf = S::NB == 2 ? 2 * m + (x & 1) : m;
        if (m == 0 && !wait(&full[v_slot], v_phase)) return;
        if (!wait(&p_full[buf], S::NB == 2 ? x >> 1 : x)) return;
        tc_fence_after();
        const uint64_t vd = v_desc + (ring_at + v_slot * (S::SLOT >> 4));
#pragma unroll
        for (int s = S::PIECES - 1; s >= 0; --s)
#pragma unroll
          for (int kk = 0; kk < S::KT / 16; ++kk)
            mma_f16_ts_elect(base + m * D, base + S::COL_S + buf * S::KT + s * (S::KT / 2) + 8 * kk, vd + (uint64_t)((kk * 2048) >> 4),
                             IDESC_O, !fresh || s != S::PIECES - 1 || kk != 0);
        if (S::NB == 2) mma_commit_elect(&o_done[m]);  // (with one buffer the next scores' commit says as much)
        if (last) mma_commit_elect(&o_last[m]);
        if (m == nm - 1) mma_commit_elect(&empty[v_slot]);
      };
      for (uint32_t m = 0; m < nm && ok; ++m)
        if (wait(&q_full[m], m ? mine1 : mine0)) issue_s(m ? cnt1 : cnt0, m);
      advance(k_slot, k_phase);
#pragma unroll 1
      for (uint32_t j = 0; j < n && ok; ++j) {
        if constexpr (S::NB == 2) {
          // chunks in order: K of tiles 0 and 1, V of tile 0, K of tile 2, V of tile 1, ...
          v_slot = k_slot, v_phase = k_phase;
          if (j + 1 < n) advance(v_slot, v_phase);
          for (uint32_t m = 0; m < nm && ok; ++m) {
            const uint32_t x = (m ? cnt1 : cnt0) + j;
            if (j + 1 < n) issue_s(x + 1, m);
            if (ok) issue_o(x, m, S::TWO ? j % S::FOLD_TILES == 0 : j == 0, j + 1 == n);
          }
          k_slot = v_slot, k_phase = v_phase;
          advance(k_slot, k_phase);
        } else {
          // K of tile 0, V of tile 0, K of tile 1, ...; one M tile's products while the other's softmax runs
          v_slot = k_slot, v_phase = k_phase;
          advance(k_slot, k_phase);
          for (uint32_t m = 0; m < nm && ok; ++m) {
            const uint32_t x = (m ? cnt1 : cnt0) + j;
            issue_o(x, m, S::TWO ? j % S::FOLD_TILES == 0 : j == 0, j + 1 == n);
            if (ok && j + 1 < n) issue_s(x + 1, m);
          }
          if (j + 1 < n) advance(k_slot, k_phase);
        }
      }
      cnt0 += n, ++mine0;
      if (nm == 2) cnt1 += n, ++mine1;
      if (!ok) break;
    }
    // the products in flight have finished before tensor memory goes
    mma_commit_elect(&drain);
    __all_sync(0xffffffffu, mbar_wait(&drain, 0, abort_flag + 1, v.status));
  } else if (warp == PIECE_WARP) {
    // ------------------------------------------------ the pieces of the share, and their cuts, ahead of the others
    Pieces<S> pieces{s_found_b, idle ? 0 : u, idle ? 0 : u_end, s_found[0], share, total};
    int4 record = make_int4(0, 0, 0, 0);
    Piece p;
    p.k1 = p.to = 0;
    bool more = true;
    for (int ip = 0; more && wait_piece(&piece_empty[ip & 1], (ip >> 1) + 1); ++ip) {
      if (p.k1 < p.to) {
        p.k0 = p.k1;
      } else {
        int t, made_of;
        more = pieces.next(a, p, t, made_of);
        if (more && made_of > 1) record = make_int4(p.b, t, p.g, made_of);
      }
      p.k1 = !more ? 0 : (S::TWO ? p.to : min(p.k0 + S::FOLD_TILES, p.to));
      if (lane == 0) {
        s_piece[ip & 1] = p;
        mbar_arrive(&piece_full[ip & 1]);
      }
      __syncwarp();
    }
    if (lane == 0) a.record[blockIdx.x] = record;
  } else if (warp == COPY_WARP) {
    // ------------------------------------------------ chunks of codes, page by page, in the order in which they are used
    const int run = min(1 << v.page_shift, S::KT);  // positions of a tile that lie together
    uint32_t sent = 0;
    for (int ip = 0; piece_is(ip); piece_done(ip), ++ip) {
      const Piece& p = s_piece[ip & 1];
      const int n = p.k1 - p.k0, k0 = p.k0, len = p.len;
      auto at_of = [&](int group) { return group_at(a, p, group); };
      Window<uint32_t, decltype(at_of)> k_at, v_at;
      k_at.begin(k0 * S::GROUPS, at_of);
      v_at = k_at;
      auto send = [&](int j, const int8_t* codes, Window<uint32_t, decltype(at_of)>& at) {
        const int tile = k0 + j, rs = sent % S::RAWS;
        at.reach(tile * S::GROUPS, at_of);
        const int first = lane * run, pos = tile * S::KT + first;  // this lane's positions of the tile
        const uint32_t g = __shfl_sync(0xffffffffu, at.now, min(tile * S::GROUPS + first / 32 - at.base, 31));
        const bool some = first < S::KT && pos < len;  // (what lies past the sequence stays as it was: any codes are numbers)
        const int runs = __popc(__ballot_sync(0xffffffffu, some));
        if (!wait(&raw_empty[rs], sent / S::RAWS + 1)) return;
        if (lane == 0) {
          if (runs > 0)
            mbar_arrive_expect_tx(&raw_full[rs], (uint32_t)(runs * run * D));
          else
            mbar_arrive(&raw_full[rs]);
        }
        __syncwarp();
        if (some) bulk_load_1d(raw + rs * S::RAW + first * D, codes + (size_t)g * 32 * D, (uint32_t)(run * D), &raw_full[rs]);
        ++sent;
      };
      // (in the order of the products)
      if (S::NB == 2) send(0, v.K, k_at);
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j) {
        if (S::NB == 1) send(j, v.K, k_at);
        if (S::NB == 2 && j + 1 < n) send(j + 1, v.K, k_at);
        if (ok) send(j, v.V, v_at);
      }
      if (!ok) break;
    }
    if (!ok)  // the copies on their way land before the CTA ends
      for (uint32_t i = sent > (uint32_t)S::RAWS ? sent - S::RAWS : 0; i < sent; ++i)
        mbar_wait(&raw_full[i % S::RAWS], (i / S::RAWS) & 1, abort_flag + 1, v.status);
  }
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- the pieces
// The segment that CTA blockIdx.x began and others ended: its pieces' outputs by their totals, in order. 32
// dims of 128 pairs a CTA (with 8, four times as many that mostly find nothing to do, 4 us more for 512 rows over 2048).
constexpr int JOIN_THREADS = 256;

template <typename T, int D>
__global__ void __launch_bounds__(JOIN_THREADS) kv8_prefill_combine_kernel(const __grid_constant__ PrefillArgs a) {
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
  // (several pieces' loads are on their way together)
  float top = -INFINITY;
#pragma unroll 8
  for (int i = 0; i < rec.w; ++i) {
    const float2 ml = a.part_ml[slot(i) * S::PAIRS + r];
    top = ml.y != 0.f ? fmaxf(top, ml.x) : top;
  }
  float all = 0.f;
#pragma unroll 8
  for (int i = 0; i < rec.w; ++i) {
    const float2 ml = a.part_ml[slot(i) * S::PAIRS + r];
    all += ml.y != 0.f ? ml.y * exp2f(ml.x - top) : 0.f;
  }
  const float inv = all == 0.f ? 0.f : 1.f / all;
  float4 y[4] = {};
#pragma unroll 4
  for (int i = 0; i < rec.w; ++i) {
    const float2 ml = a.part_ml[slot(i) * S::PAIRS + r];
    const float4* o = a.part_o + (slot(i) * (D / 4) + c0) * S::PAIRS + r;
    float4 x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = o[(size_t)c * S::PAIRS];
    const float f = ml.y != 0.f ? ml.y * exp2f(ml.x - top) * inv : 0.f;  // (at most 1: no sum of large values leaves the range)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      y[c].x = fmaf(x[c].x, f, y[c].x), y[c].y = fmaf(x[c].y, f, y[c].y), y[c].z = fmaf(x[c].z, f, y[c].z), y[c].w = fmaf(x[c].w, f, y[c].w);
  }
  const int i = (int)quotient(pair, a.group);
  T* to = static_cast<T*>(a.out) + (long long)(w.r0 + i) * a.ldo + ((size_t)rec.z * a.group + (size_t)(pair - (long long)i * a.group)) * D + 4 * c0;
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
  cfg.blockDim = dim3(JOIN_THREADS);
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

size_t kv8_prefill_scratch(const Kv8View& v) {
  return (size_t)num_sms() * (16 + 3 * (piece_bytes(v.dim) + pairs_of(v.dim) * 8));
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
  at += ctas * 16;
  a.mean_ml = reinterpret_cast<float2*>(at);
  a.mean = reinterpret_cast<float4*>(at + ctas * pairs_of(v.dim) * 8);
  if (type == APR_T_F32) return launch_typed<float>(a, s);
  if (type == APR_T_F16) return launch_typed<__half>(a, s);
  return launch_typed<__nv_bfloat16>(a, s);
}

}  // namespace apr
