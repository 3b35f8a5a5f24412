// k and v rows into the 8-bit paged KV cache, k normed and rotated on the way, q rotated
// beside them (include/apr_rope.h): one launch between a chunk's qkv projection and its
// attention, in which every row is read once.
//
// The append's CTAs are those of kv8_append.cu, a page of some heads, K or V; a K
// vector is a unit of four pairs (rope.cuh), so a rotation stays within its thread and a
// head's mean of squares within D / 8 neighbouring lanes. What is quantised are the values
// rounded to the rows' type, the bits that apr_rope_rows would have written. The CTAs behind them
// rotate the q rows.
//
// Bound by latency at 24 warps an SM: a head is loaded, normed and rotated, its largest magnitude found across a barrier, and quantised
// before the next head's loads begin (63 % of the issue slots taken, HBM at 0.4 of its rate, loads the largest stall). 13157 bf16 rows of 8
// normed heads of 128 on three axes take 49 us (61 with K's CTAs among V's, whose last ones ended late), 89 with 32 heads of q (156 before a page's
// turns were looked up once and a head's rows kept); 50001 fp16 rows of 8 heads of 64 63 us, 92 with 16 of q; 64 rows 5.0 and 6.6 us; 8192
// float32 rows of 4 normed heads of 256 28 us in pages of 64 (33 if they are not kept, below), 33 in pages of 128, 48 in pages of 256; with 16
// heads of q 79, 83 and 83.

#include "apr_internal.h"
#include "host_common.h"
#include "kv8_append.cuh"
#include "rope.cuh"

namespace apr {
namespace {

// K's CTAs of an SM that the heads are divided for, where each looks its page's turns up first (13157 rows with q 89 us, 90 with 8, 92 with
// 12; without q 49, 42 with 8; but 8192 float32 rows of 8 heads of 128 without q 48, 58 with 8, and with 32 heads of q 128 and 138).
constexpr int K_CTAS = 5;

struct AppendArgs {
  Kv8View v;
  RopeView r;
  const void* k;
  const void* vv;
  long long ld;
  const float* k_norm;
  float eps;
  int k_heads, v_heads;  // that a CTA takes one after the other
  unsigned k_ctas;       // the first ones: they take longest
  unsigned append_ctas;  // with V's; the CTAs behind them are q's
  int staged;            // bytes of a page's cosines and sines, where they are looked up once for all heads
  int kept;              // a head's rows fit shared memory, and are not loaded, normed and rotated twice
  RopeRows q;            // heads 0: none
};

// TH threads: 128 where a page's rows have no more units.
template <typename T, int D, int TH>
__global__ void __launch_bounds__(TH, TH == 128 ? 4 : (sizeof(T) == 4 ? 2 : 3)) kv8_append_rope_kernel(const __grid_constant__ AppendArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  extern __shared__ __align__(16) uint8_t smem[];  // [rows][pairs] cosines, then sines; a head's rows
  const Kv8View& v = a.v;
  constexpr int ROW = D / 8;  // units of a head, and lanes of a group
  if (blockIdx.x >= a.append_ctas) {
    const long long group = (long long)(blockIdx.x - a.append_ctas) * (TH / ROW) + threadIdx.x / ROW;
    const int row = (int)min(rope_row_of(a.q, group), (long long)v.num_rows - 1);
    // rows ahead of the first sequence's and behind the last one's are nobody's
    const bool live = !v.row_start || (row >= v.row_start[0] && row < v.row_start[v.num_seqs]);
    int own = 0;
    if (live && !a.r.positions) {  // the row's position in its sequence: the last one that begins at the row or before it
      int b = row;
      if (v.row_start) {
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
      const Kv8Span span = kv8_rows(v, b);
      own = row >= span.r0 && row < span.r0 + span.n ? kv8_len(v, b) - span.n + row - span.r0 : 0;
    }
    rope_rows_group<T, ROW, 1>(a.r, a.q, group, threadIdx.x % ROW, own, live);
    return;
  }
  const bool is_v = blockIdx.x >= a.k_ctas;
  const int each = is_v ? a.v_heads : a.k_heads, parts = (v.kv_heads + each - 1) / each, cta = (int)(blockIdx.x - (is_v ? a.k_ctas : 0));
  const int index_of_unit = cta / parts, part = cta % parts;
  constexpr int STEP = TH / ROW;  // rows from one of a thread's vectors to the next
  __shared__ float s_max[3][TH / 32];
  const int g0 = part * each, g1 = min(g0 + each, v.kv_heads);

  // ---- which page: the slot-th that the sequence's rows go to, if it has so many
  int b = index_of_unit, slot = 0;
  if (v.row_start) {
    b = kv8_last_sequence(v, [&](int i) { return first_append_unit(v, i) <= index_of_unit; });
    slot = index_of_unit - first_append_unit(v, b);
    // every length and range is looked at, also one that no unit is found by
    if (!is_v && part == 0 && index_of_unit < v.num_seqs && threadIdx.x == 0) kv8_len(v, index_of_unit), kv8_rows(v, index_of_unit);
  }
  const int len = kv8_len(v, b);
  const Kv8Span span = kv8_rows(v, b);
  const int first = len - span.n;  // position of row r0; rows of negative positions are skipped
  const int index = (max(first, 0) >> v.page_shift) + slot;
  if (slot < 0 || span.n == 0 || len == 0 || index > (len - 1) >> v.page_shift) return;
  const int page = v.table[(size_t)b * v.table_ld + index];
  if (page < 0 || page >= v.num_pages) {
    if (threadIdx.x == 0) kv8_flag(v);
    return;
  }
  const int page0 = index << v.page_shift;
  const int lo = max(max(first, 0), page0), hi = min(len, page0 + (1 << v.page_shift));
  const int held = lo - page0;
  const int nvec = (hi - lo) * ROW;
  // this thread's vectors: one unit, every STEP-th row
  const int u = (int)threadIdx.x % ROW, row0 = (int)threadIdx.x / ROW;
  const RopeUnit unit = is_v ? RopeUnit{8 * u, 8 * u + 4, -1, 0} : rope_unit(a.r, u);
  const bool normed = !is_v && a.k_norm;
  float w[8];
  if (normed) {
    const Vec8<float> x = load44(a.k_norm, unit.d0, unit.d1);
    values8(x, w);
  }
  const T* src = static_cast<const T*>(is_v ? a.vv : a.k) + (long long)(span.r0 + lo - first + row0) * a.ld + (size_t)g0 * D;
  const int rows = hi - lo;
  float* s_turn = reinterpret_cast<float*>(smem);
  Vec8<T>* s_rows = reinterpret_cast<Vec8<T>*>(smem + a.staged);
  const bool staged = !is_v && a.staged;
  if (staged) {
    // the page's cosines and sines, for all the heads
    // (a thread a pair, every few rows)
    const int pairs = a.r.pairs, i = (int)threadIdx.x % pairs, step = TH / pairs;
    int axis = a.r.axis ? a.r.axis[i] : 0;
    if (axis >= a.r.num_axes) axis = 0;  // (flagged by rope_unit)
    const float2* column = a.r.table + i;
    if ((int)threadIdx.x < step * pairs) {
      bool bad = false;
      for (int row0 = (int)threadIdx.x / pairs; row0 < rows; row0 += 8 * step) {
        float2 t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = min(row0 + k * step, rows - 1);
          t[k] = column[(size_t)rope_position(a.r, axis, span.r0 + lo - first + row, lo + row, bad) * pairs];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = row0 + k * step;
          if (row < rows) {
            s_turn[row * pairs + i] = t[k].x;
            s_turn[(rows + row) * pairs + i] = t[k].y;
          }
        }
      }
      if (bad) atomicOr(a.r.status, kStatusBadIndex);
    }
    __syncthreads();
  }
  // vector j's cosines and sines
  auto turn_of = [&](int j) -> RopeTurn {
    const int row = row0 + j * STEP;
    if (!staged) return rope_turn(a.r, unit, span.r0 + lo - first + row, lo + row);
    const float4 c = *reinterpret_cast<const float4*>(s_turn + row * a.r.pairs + unit.pair);
    const float4 t = *reinterpret_cast<const float4*>(s_turn + (rows + row) * a.r.pairs + unit.pair);
    return RopeTurn{{make_float2(c.x, t.x), make_float2(c.y, t.y), make_float2(c.z, t.z), make_float2(c.w, t.w)}};
  };
  auto is_live = [&](int j) { return (int)threadIdx.x + j * TH < nvec; };
  // vectors j .. j + 3 of a head as they go into the cache
  auto vectors = [&](int j, const T* from, Vec8<T> (&e)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[i] = ones8<T>();
      if (is_live(j + i)) e[i] = load44(from + (long long)(j + i) * STEP * a.ld, unit.d0, unit.d1);
    }
    if (is_v) return;
    float inv[4];
    if (normed) {
      HeadPart<T, 1> part[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) part[i].v[0] = e[i];
      rope_inverse_rms4_of_any<ROW>(part, (float)D, 1.f / D, a.eps, inv);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!is_live(j + i)) continue;
      float x[8];
      values8(e[i], x);
      if (normed) rope_norm(x, inv[i], w);
      if (unit.pair >= 0) rope_rotate(a.r, unit, turn_of(j + i), x);
      e[i] = vec8_of<T>(x);
    }
  };
  int8_t* codes = (is_v ? v.V : v.K) + kv8_codes_at(v, page, g0);
  float* scale = (is_v ? v.v_scale : v.k_scale) + kv8_scale_at(v, page, g0);
  for (int g = g0; g < g1; ++g, src += D, codes += (size_t)D << v.page_shift, ++scale) {
    const float s_old = held > 0 ? *scale : 0.f;
    // ---- the largest magnitude
    float m = 0.f;
#pragma unroll 1
    for (int j = 0; j * TH < nvec; j += 4) {
      Vec8<T> e[4];
      vectors(j, src, e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (is_live(j + i)) {
          m = amax_of(e[i], m);
          if (a.kept) s_rows[(j + i) * TH + threadIdx.x] = e[i];
        }
    }
    m = block_max<TH / 32>(m, s_max[g & 1]);  // (the next head writes the other: one barrier a head)
    if (m > FLT_MAX) {                        // an infinity among them, for the whole CTA
      m = 0.f;
#pragma unroll 1
      for (int j = 0; j * TH < nvec; j += 4) {
        Vec8<T> e[4];
        vectors(j, src, e);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (is_live(j + i)) m = finite_amax_of<T>(e[i], m);
      }
      __syncthreads();
      m = block_max<TH / 32>(m, s_max[2]);
    }

    // ---- the scale, and what the page held under a raised one
    const Kv8Scale s = kv8_rounding_to(fmaxf(s_old, kv8_scale_of(m)));
    if (threadIdx.x == 0 && (held == 0 || s.s > s_old)) *scale = s.s;
    if (held > 0 && s.s > s_old) {
      uint4* old = reinterpret_cast<uint4*>(codes);
      for (int i = threadIdx.x; i < held * D / 16; i += TH) {
        const uint4 x = old[i];
        uint4 y = kv8_requantise16(x, s_old, s);
        // (a code of -128 may have come from elsewhere)
        y.x = __vmaxs4(y.x, 0x81818181u), y.y = __vmaxs4(y.y, 0x81818181u);
        y.z = __vmaxs4(y.z, 0x81818181u), y.w = __vmaxs4(y.w, 0x81818181u);
        old[i] = y;
      }
    }

    // ---- the new codes
    int8_t* dst = codes + (size_t)(held + row0) * D;
    auto store = [&](int j, const Vec8<T>& e) {
      const uint2 c = codes_of<T>(e, s);
      int8_t* p = dst + (size_t)j * STEP * D;
      *reinterpret_cast<uint32_t*>(p + unit.d0) = c.x;
      *reinterpret_cast<uint32_t*>(p + unit.d1) = c.y;
    };
#pragma unroll 1
    for (int j = 0; j * TH < nvec; j += 4) {
      Vec8<T> e[4];
      if (a.kept) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (is_live(j + i)) e[i] = s_rows[(j + i) * TH + threadIdx.x];
      } else {
        vectors(j, src, e);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (is_live(j + i)) store(j + i, e[i]);
    }
  }
}

template <typename T, int D, int TH>
cudaError_t append_shape(AppendArgs& a, cudaStream_t s) {
  const Kv8View& v = a.v;
  // the most pages that the rows can touch (first_append_unit)
  const long long pages = v.row_start ? (v.num_rows >> v.page_shift) + 2ll * v.num_seqs : v.num_seqs;
  // the turns of a page's rows, but no more rows than a sequence has
  const size_t rows = v.max_rows < 1 << v.page_shift ? v.max_rows : 1 << v.page_shift;
  const size_t turns = rows * a.r.pairs * 8, held = rows * D * sizeof(T);
  a.staged = rows >= 16 && turns <= 64 * 1024 && v.kv_heads > 1 ? (int)turns : 0;
  // (kept up to 64 KB, normed rows of 4 heads of 256 without q: 8192 float32 ones in pages of 64 28 us, 33 if not; bf16 ones in pages of 128
  // 29 and 37. With q, whose CTAs have the same shared memory: 79 and 83, 70 and 63, but 128 and 86 for float32 rows of 8 + 32
  // heads of 128 in pages of 128, whose turns take another 64 KB. Past 64 KB a CTA an SM is left: 82 us become 122, 71 become 111)
  a.kept = held <= 64 * 1024;
  a.v_heads = heads_a_cta(pages, v.kv_heads, 12);
  a.k_heads = a.staged ? heads_a_cta(pages, v.kv_heads, K_CTAS) : a.v_heads;
  a.k_ctas = (unsigned)(pages * ((v.kv_heads + a.k_heads - 1) / a.k_heads));
  a.append_ctas = a.k_ctas + (unsigned)(pages * ((v.kv_heads + a.v_heads - 1) / a.v_heads));
  constexpr int GROUPS = TH / (D / 8);
  long long q_ctas = 0;
  if (a.q.heads > 0) {
    a.q.heads_a_group = rope_heads_a_group(v.num_rows, a.q.heads, GROUPS * 8ll * num_sms());
    q_ctas = ((long long)v.num_rows * ((a.q.heads + a.q.heads_a_group - 1) / a.q.heads_a_group) + GROUPS - 1) / GROUPS;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.append_ctas + q_ctas));
  cfg.blockDim = dim3(TH);
  cfg.dynamicSmemBytes = (a.staged ? turns : 0) + (a.kept ? held : 0);
  if (cfg.dynamicSmemBytes > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kv8_append_rope_kernel<T, D, TH>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    if (e != cudaSuccess) return e;
  }
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_append_rope_kernel<T, D, TH>, a);
}
template <typename T, int D>
cudaError_t append_sized(AppendArgs& a, cudaStream_t s) {
  return a.v.max_rows * (D / 8) <= 128 ? append_shape<T, D, 128>(a, s) : append_shape<T, D, 256>(a, s);
}
template <typename T>
cudaError_t append_typed(AppendArgs& a, cudaStream_t s) {
  return a.v.dim == 64 ? append_sized<T, 64>(a, s) : (a.v.dim == 128 ? append_sized<T, 128>(a, s) : append_sized<T, 256>(a, s));
}

}  // namespace

cudaError_t launch_rope_kv8_append(const Kv8View& v, const RopeView& r, int type, const void* k, const void* vv,
                                   long long ld, const float* k_norm, float eps, const RopeRows& q, cudaStream_t s) {
  AppendArgs a{v, r, k, vv, ld, k_norm, eps, 0, 0, 0, 0, 0, 0, q};
  if (type == APR_T_F32) return append_typed<float>(a, s);
  if (type == APR_T_F16) return append_typed<__half>(a, s);
  return append_typed<__nv_bfloat16>(a, s);
}

}  // namespace apr
