// k and v rows into the 8-bit paged KV cache, k normed and rotated on the way, q rotated
// beside them (include/apr_rope.h): one launch between a chunk's qkv projection and its
// attention, in which every row is read once.
//
// The append's CTAs are those of kv8_append.cu, a page of some heads, K or V; a K
// vector is a unit of four pairs (rope.cuh), so a rotation stays within its thread and a
// head's mean of squares within D / 8 neighbouring lanes. What is quantised are the values
// rounded to the rows' type, the bits that apr_rope_rows would have written. The CTAs behind them
// rotate the q rows.

#include "apr_internal.h"
#include "host_common.h"
#include "kv8_append.cuh"
#include "rope.cuh"

namespace apr {
namespace {

struct AppendArgs {
  Kv8View v;
  RopeView r;
  const void* k;
  const void* vv;
  long long ld;
  const float* k_norm;
  float eps;
  int heads_a_cta;
  unsigned append_ctas;  // the CTAs behind them are q's
  RopeRows q;            // heads 0: none
};

template <typename T, int D>
__global__ void __launch_bounds__(A_THREADS, 4) kv8_append_rope_kernel(const __grid_constant__ AppendArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const Kv8View& v = a.v;
  constexpr int ROW = D / 8;  // units of a head, and lanes of a group
  if (blockIdx.x >= a.append_ctas) {
    const long long group = (long long)(blockIdx.x - a.append_ctas) * (A_THREADS / ROW) + threadIdx.x / ROW;
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
  const int parts = 2 * ((v.kv_heads + a.heads_a_cta - 1) / a.heads_a_cta);
  const int index_of_unit = (int)(blockIdx.x / parts), part = (int)(blockIdx.x % parts);
  constexpr int HELD = 16 / sizeof(T);  // vectors of 8 values a thread keeps between the passes, 32 registers
  constexpr int STEP = A_THREADS / ROW;  // rows from one of a thread's vectors to the next
  __shared__ float s_max[3][A_WARPS];
  const bool is_v = part & 1;
  const int g0 = (part >> 1) * a.heads_a_cta, g1 = min(g0 + a.heads_a_cta, v.kv_heads);

  // ---- which page: the slot-th that the sequence's rows go to, if it has so many
  int b = index_of_unit, slot = 0;
  if (v.row_start) {
    b = kv8_last_sequence(v, [&](int i) { return first_append_unit(v, i) <= index_of_unit; });
    slot = index_of_unit - first_append_unit(v, b);
    // every length and range is looked at, also one that no unit is found by
    if (part == 0 && index_of_unit < v.num_seqs && threadIdx.x == 0) kv8_len(v, index_of_unit), kv8_rows(v, index_of_unit);
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
  const int nvec_all = (nvec + 31) & ~31;  // whole warps go through a norm together
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
  // vector j of head g as it goes into the cache
  auto vector = [&](int j, const T* from) -> Vec8<T> {
    Vec8<T> e = {};
    const bool live = (int)threadIdx.x + j * A_THREADS < nvec;
    if (live) e = load44(from + (long long)j * STEP * a.ld, unit.d0, unit.d1);
    if (is_v) return e;
    float x[8];
    values8(e, x);
    if (normed) {
      rope_norm(x, rope_inverse_rms(two_group_sum<ROW>(squares_of<sizeof(T) == 2>(x)), (float)D, 1.f / D, a.eps), w);
    }
    if (live && unit.pair >= 0) {
      const int pos = lo + row0 + j * STEP;
      rope_rotate(a.r, unit, rope_turn(a.r, unit, span.r0 + pos - first, pos), x);
    }
    return vec8_of<T>(x);
  };
  int8_t* codes = (is_v ? v.V : v.K) + kv8_codes_at(v, page, g0);
  float* scale = (is_v ? v.v_scale : v.k_scale) + kv8_scale_at(v, page, g0);
  for (int g = g0; g < g1; ++g, src += D, codes += (size_t)D << v.page_shift, ++scale) {
    const float s_old = held > 0 ? *scale : 0.f;
    // ---- the largest magnitude
    Vec8<T> keep[HELD];
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < HELD; ++j)
      if ((int)threadIdx.x + j * A_THREADS < nvec_all) {
        keep[j] = vector(j, src);
        if ((int)threadIdx.x + j * A_THREADS < nvec) m = amax_of(keep[j], m);
      }
    for (int j = HELD; (int)threadIdx.x + j * A_THREADS < nvec_all; ++j) {
      const Vec8<T> e = vector(j, src);
      if ((int)threadIdx.x + j * A_THREADS < nvec) m = amax_of(e, m);
    }
    m = block_max<A_WARPS>(m, s_max[g & 1]);  // (the next head writes the other: one barrier a head)
    if (m > FLT_MAX) {                        // an infinity among them, for the whole CTA
      m = 0.f;
      for (int j = 0; (int)threadIdx.x + j * A_THREADS < nvec_all; ++j) {
        const Vec8<T> e = vector(j, src);
        if ((int)threadIdx.x + j * A_THREADS < nvec) m = finite_amax_of<T>(e, m);
      }
      __syncthreads();
      m = block_max<A_WARPS>(m, s_max[2]);
    }

    // ---- the scale, and what the page held under a raised one
    const Kv8Scale s = kv8_rounding_to(fmaxf(s_old, kv8_scale_of(m)));
    if (threadIdx.x == 0 && (held == 0 || s.s > s_old)) *scale = s.s;
    if (held > 0 && s.s > s_old) {
      uint4* old = reinterpret_cast<uint4*>(codes);
      for (int i = threadIdx.x; i < held * D / 16; i += A_THREADS) {
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
#pragma unroll
    for (int j = 0; j < HELD; ++j)
      if ((int)threadIdx.x + j * A_THREADS < nvec) store(j, keep[j]);
    for (int j = HELD; (int)threadIdx.x + j * A_THREADS < nvec_all; ++j) {
      const Vec8<T> e = vector(j, src);
      if ((int)threadIdx.x + j * A_THREADS < nvec) store(j, e);
    }
  }
}

template <typename T, int D>
cudaError_t append_shape(AppendArgs& a, cudaStream_t s) {
  const Kv8View& v = a.v;
  // the most pages that the rows can touch (first_append_unit)
  const long long pages = v.row_start ? (v.num_rows >> v.page_shift) + 2ll * v.num_seqs : v.num_seqs;
  a.heads_a_cta = heads_a_cta(pages, v.kv_heads, 12);
  a.append_ctas = (unsigned)(pages * 2 * ((v.kv_heads + a.heads_a_cta - 1) / a.heads_a_cta));
  constexpr int GROUPS = A_THREADS / (D / 8);
  long long q_ctas = 0;
  if (a.q.heads > 0) {
    a.q.heads_a_group = a.q.heads < 4 ? a.q.heads : 4;
    q_ctas = ((long long)v.num_rows * ((a.q.heads + a.q.heads_a_group - 1) / a.q.heads_a_group) + GROUPS - 1) / GROUPS;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.append_ctas + q_ctas));
  cfg.blockDim = dim3(A_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_append_rope_kernel<T, D>, a);
}
template <typename T>
cudaError_t append_typed(AppendArgs& a, cudaStream_t s) {
  return a.v.dim == 64 ? append_shape<T, 64>(a, s) : (a.v.dim == 128 ? append_shape<T, 128>(a, s) : append_shape<T, 256>(a, s));
}

}  // namespace

cudaError_t launch_rope_kv8_append(const Kv8View& v, const RopeView& r, int type, const void* k, const void* vv,
                                   long long ld, const float* k_norm, float eps, const RopeRows& q, cudaStream_t s) {
  AppendArgs a{v, r, k, vv, ld, k_norm, eps, 0, 0, q};
  if (type == APR_T_F32) return append_typed<float>(a, s);
  if (type == APR_T_F16) return append_typed<__half>(a, s);
  return append_typed<__nv_bfloat16>(a, s);
}

}  // namespace apr
