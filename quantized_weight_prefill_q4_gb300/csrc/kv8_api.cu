// C ABI of the 8-bit paged KV cache (include/apr_kv8.h) and of the rotations by
// position (include/apr_rope.h): argument checks, scratch, launches.

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <exception>

#include "apr_internal.h"
#include "apr_kv8.h"
#include "apr_rope.h"
#include "kv8.cuh"
#include "rope.cuh"

using namespace apr;

namespace {

int failf(int code, const char* fmt, long long a = 0, long long b = 0, long long c = 0) {
  char msg[256];
  snprintf(msg, sizeof msg, fmt, a, b, c);
  return set_error(code, msg);
}

bool on16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool on4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return na && nb && a0 < b0 + nb && b0 < a0 + na;
}
int type_size(int type) { return type == APR_T_F32 ? 4 : (type == APR_T_F16 || type == APR_T_BF16 ? 2 : 0); }

// One element range of an argument, for the overlap checks.
struct Range {
  const void* p;
  size_t bytes;
  const char* name;
};
// Elements of `count` rows of `width` every `ld`.
size_t span_of(long long count, long long ld, long long width) {
  return count > 0 ? (size_t)(count - 1) * (size_t)ld + (size_t)width : 0;
}

// Whether `count` rows of wa bytes every lda from a and as many of wb bytes every ldb from b meet. Of one distance
// they may be slices of one buffer, rows that interleave; of two, their whole ranges count.
bool rows_meet(const void* a, size_t lda, size_t wa, const void* b, size_t ldb, size_t wb, long long count) {
  if (!meet(a, span_of(count, lda, wa), b, span_of(count, ldb, wb))) return false;
  if (lda != ldb) return true;
  const bool a_first = (uintptr_t)a <= (uintptr_t)b;
  const size_t off = (a_first ? (uintptr_t)b - (uintptr_t)a : (uintptr_t)a - (uintptr_t)b) % lda;
  return off < (a_first ? wa : wb) || lda - off < (a_first ? wb : wa);
}

// Checks the cache and the rows, and fills the kernels' view of them. Returns
// APR_OK, an error, or 1 where there is nothing to do: no sequences, or no rows
// (unless `per_seq`: the call writes something for each sequence all the same).
int view_of(const apr_kv8_cache* c, const apr_kv8_rows* r, bool with_rows, bool per_seq, Kv8View* v) {
  if (!c || !r) return set_error(APR_E_INVAL, "null cache or rows");
  if (c->num_pages < 1 || c->num_pages > (1 << 27) || c->num_kv_heads < 1 || c->num_kv_heads > 1024)
    return failf(APR_E_INVAL, "bad cache: num_pages=%lld num_kv_heads=%lld", c->num_pages, c->num_kv_heads);
  if (c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128 && c->page_tokens != 256)
    return failf(APR_E_INVAL, "page_tokens must be 32, 64, 128 or 256 (got %lld)", c->page_tokens);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return failf(APR_E_INVAL, "head_dim must be 64, 128 or 256 (got %lld)", c->head_dim);
  if ((long long)c->num_pages * c->num_kv_heads * c->page_tokens > (1LL << 36))
    return set_error(APR_E_INVAL, "a cache of more than 2^36 tokens and heads");
  if (r->num_seqs < 0 || r->num_seqs > 16384 || r->num_rows < 0 || r->num_rows > (1 << 24))
    return failf(APR_E_INVAL, "bad sizes: num_seqs=%lld num_rows=%lld", r->num_seqs, r->num_rows);
  if (with_rows && !r->row_start && r->num_rows != r->num_seqs)
    return failf(APR_E_INVAL, "without row_start there is one row a sequence: num_rows=%lld, num_seqs=%lld",
                 r->num_rows, r->num_seqs);
  const long long cap = (long long)r->table_ld * c->page_tokens;
  if (r->table_ld < 0 || cap > (1LL << 30)) return failf(APR_E_INVAL, "bad table_ld=%lld", r->table_ld);
  if (r->max_len < 0 || r->max_len > cap)
    return failf(APR_E_INVAL, "max_len=%lld is not within the table's %lld tokens", r->max_len, cap);
  if (r->max_rows < 0 || (with_rows && r->max_rows > r->num_rows))
    return failf(APR_E_INVAL, "max_rows=%lld is not within num_rows=%lld", r->max_rows, r->num_rows);
  if (r->num_seqs == 0 || (with_rows && !per_seq && r->num_rows == 0)) return 1;
  if (!c->K || !c->V || !c->k_scale || !c->v_scale) return set_error(APR_E_INVAL, "null pointer in the cache");
  if (!r->lens || (!r->page_table && r->table_ld > 0)) return set_error(APR_E_INVAL, "null page_table or lens");
  if (!on16(c->K) || !on16(c->V)) return set_error(APR_E_ALIGN, "the cache's codes are not 16-byte aligned");
  if (!on4(c->k_scale) || !on4(c->v_scale) || !on4(r->page_table) || !on4(r->lens) || !on4(r->row_start))
    return set_error(APR_E_ALIGN, "scales, page_table, lens or row_start are not 4-byte aligned");
  const size_t scales = (size_t)c->num_pages * c->num_kv_heads;
  const size_t codes = scales * c->page_tokens * c->head_dim;
  if (meet(c->K, codes, c->V, codes) || meet(c->k_scale, scales * 4, c->v_scale, scales * 4) ||
      meet(c->K, codes, c->k_scale, scales * 4) || meet(c->K, codes, c->v_scale, scales * 4) ||
      meet(c->V, codes, c->k_scale, scales * 4) || meet(c->V, codes, c->v_scale, scales * 4))
    return set_error(APR_E_ALIAS, "the cache's arrays overlap");
  v->K = reinterpret_cast<int8_t*>(c->K);
  v->V = reinterpret_cast<int8_t*>(c->V);
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  v->table = r->page_table;
  v->lens = r->lens;
  v->row_start = with_rows ? r->row_start : nullptr;
  v->status = nullptr;
  v->num_pages = c->num_pages;
  v->kv_heads = c->num_kv_heads;
  v->page_shift = c->page_tokens == 32 ? 5 : (c->page_tokens == 64 ? 6 : (c->page_tokens == 128 ? 7 : 8));
  v->dim = c->head_dim;
  v->table_ld = r->table_ld;
  v->num_seqs = r->num_seqs;
  v->num_rows = r->num_rows;
  v->max_rows = !with_rows ? 0 : (r->row_start ? (r->max_rows ? r->max_rows : r->num_rows) : 1);
  v->max_len = r->max_len ? r->max_len : (int)cap;
  return APR_OK;
}

// The first of `ins` that one of `outs` overlaps gives APR_E_ALIAS; so do two
// outputs that overlap.
template <int N, int M>
int check_overlap(const Range (&outs)[N], const Range (&ins)[M]) {
  char msg[160];
  for (int i = 0; i < N; ++i) {
    for (const Range& in : ins)
      if (meet(outs[i].p, outs[i].bytes, in.p, in.bytes)) {
        snprintf(msg, sizeof msg, "%s overlaps %s", outs[i].name, in.name);
        return set_error(APR_E_ALIAS, msg);
      }
    for (int j = 0; j < i; ++j)
      if (meet(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) {
        snprintf(msg, sizeof msg, "%s overlaps %s", outs[i].name, outs[j].name);
        return set_error(APR_E_ALIAS, msg);
      }
  }
  return APR_OK;
}

size_t code_bytes(const Kv8View& v) { return ((size_t)v.num_pages * v.kv_heads << v.page_shift) * v.dim; }
size_t scale_bytes(const Kv8View& v) { return (size_t)v.num_pages * v.kv_heads * 4; }
size_t table_bytes(const Kv8View& v) { return (size_t)v.num_seqs * v.table_ld * 4; }
size_t start_bytes(const Kv8View& v) { return v.row_start ? ((size_t)v.num_seqs + 1) * 4 : 0; }

// The k and v rows of the append and the read.
int check_rows(const Kv8View& v, int type, const void* k, const void* vv, long long ld) {
  const int size = type_size(type);
  if (!size) return failf(APR_E_INVAL, "unknown element type %lld", type);
  const long long width = (long long)v.kv_heads * v.dim;
  if (ld < width || ld > (1LL << 28))
    return failf(APR_E_INVAL, "ld=%lld must be within num_kv_heads * head_dim=%lld and 2^28", ld, width);
  if (!k || !vv) return set_error(APR_E_INVAL, "null k or v");
  if (!on16(k) || !on16(vv) || ld * size % 16 != 0)
    return failf(APR_E_ALIGN, "the k and v rows (ld=%lld) are not on 16-byte boundaries", ld);
  return APR_OK;
}

// The q rows and outputs of the attentions.
int check_heads(const Kv8View& w, int type, const void* q, long long ldq, const void* out, long long ldo, int num_heads,
                float scale) {
  const int size = type_size(type);
  if (!size) return failf(APR_E_INVAL, "unknown element type %lld", type);
  if (num_heads <= 0 || num_heads > 65536 || num_heads % w.kv_heads != 0)
    return failf(APR_E_INVAL, "num_heads (%lld) must be a multiple of num_kv_heads (%lld), at most 65536", num_heads,
                 w.kv_heads);
  const long long width = (long long)num_heads * w.dim;
  if (ldq < width || ldo < width || ldq > (1LL << 28) || ldo > (1LL << 28))
    return failf(APR_E_INVAL, "ldq=%lld and ldo=%lld must be within num_heads * head_dim=%lld and 2^28", ldq, ldo,
                 width);
  if (!(scale >= 0.f) || !std::isfinite(scale)) return set_error(APR_E_INVAL, "scale must be finite and not negative");
  if (w.num_rows > 0 && (!q || !out)) return set_error(APR_E_INVAL, "null q or out");
  if (!on16(q) || !on16(out) || ldq * size % 16 != 0 || ldo * size % 16 != 0)
    return failf(APR_E_ALIGN, "the q and out rows (ldq=%lld, ldo=%lld) are not on 16-byte boundaries", ldq, ldo);
  return APR_OK;
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) return APR_OK;
  char msg[200];
  snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
  return set_error(APR_E_LAUNCH, msg);
}

int run_append(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, const void* k, const void* v,
               long long ld, cudaStream_t s) {
  Kv8View w;
  int rc = view_of(cache, rows, true, false, &w);
  if (rc != APR_OK) return rc == 1 ? APR_OK : rc;
  rc = check_rows(w, type, k, v, ld);
  if (rc != APR_OK) return rc;
  const size_t bytes = span_of(w.num_rows, ld, (long long)w.kv_heads * w.dim) * type_size(type);
  const size_t cb = code_bytes(w), sb = scale_bytes(w);
  const Range outs[] = {{w.K, cb, "K"}, {w.V, cb, "V"}, {w.k_scale, sb, "k_scale"}, {w.v_scale, sb, "v_scale"}};
  const Range ins[] = {{k, bytes, "k"},
                       {v, bytes, "v"},
                       {w.table, table_bytes(w), "page_table"},
                       {w.lens, (size_t)w.num_seqs * 4, "lens"},
                       {w.row_start, start_bytes(w), "row_start"}};
  rc = check_overlap(outs, ins);
  if (rc != APR_OK) return rc;
  rc = device_status_word(&w.status);
  if (rc != APR_OK) return rc;
  return launched(launch_kv8_append(w, type, k, v, ld, s), "append");
}

int run_read(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, void* k, void* v, long long ld,
             cudaStream_t s) {
  Kv8View w;
  int rc = view_of(cache, rows, true, false, &w);
  if (rc != APR_OK) return rc == 1 ? APR_OK : rc;
  rc = check_rows(w, type, k, v, ld);
  if (rc != APR_OK) return rc;
  const size_t width = (size_t)w.kv_heads * w.dim, size = type_size(type);
  const size_t bytes = span_of(w.num_rows, ld, width) * size;
  if (rows_meet(k, ld * size, width * size, v, ld * size, width * size, w.num_rows))
    return set_error(APR_E_ALIAS, "k overlaps v");
  const size_t cb = code_bytes(w), sb = scale_bytes(w);
  const Range ins[] = {{w.K, cb, "K"},
                       {w.V, cb, "V"},
                       {w.k_scale, sb, "k_scale"},
                       {w.v_scale, sb, "v_scale"},
                       {w.table, table_bytes(w), "page_table"},
                       {w.lens, (size_t)w.num_seqs * 4, "lens"},
                       {w.row_start, start_bytes(w), "row_start"}};
  for (const Range out : {Range{k, bytes, "k"}, Range{v, bytes, "v"}}) {
    const Range one[] = {out};
    rc = check_overlap(one, ins);
    if (rc != APR_OK) return rc;
  }
  rc = device_status_word(&w.status);
  if (rc != APR_OK) return rc;
  return launched(launch_kv8_read(w, type, k, v, ld, s), "read");
}

int run_attention(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, const void* q, long long ldq,
                  void* out, long long ldo, int num_heads, float scale, float* weights, long long weights_ld,
                  int accumulate, cudaStream_t s) {
  Kv8View w;
  int rc = view_of(cache, rows, true, weights && !accumulate, &w);
  if (rc != APR_OK) return rc == 1 ? APR_OK : rc;
  rc = check_heads(w, type, q, ldq, out, ldo, num_heads, scale);
  if (rc != APR_OK) return rc;
  const int size = type_size(type);
  const long long width = (long long)num_heads * w.dim;
  if (weights && (weights_ld < w.max_len || weights_ld > (1LL << 30)))
    return failf(APR_E_INVAL, "weights_ld=%lld must be within max_len=%lld and 2^30", weights_ld, w.max_len);
  // units of work of the kernel, counted in 32 bits (64 positions of 8 pairs of row and head)
  const long long segs = ((long long)w.num_rows * (num_heads / w.kv_heads) / 8 + w.num_seqs) * w.kv_heads;
  if (segs * (w.max_len / 64 + 10) > (1LL << 30) || (weights_ld / 128 + 1) * w.kv_heads > (1LL << 30))
    return set_error(APR_E_INVAL, "sizes beyond the supported limits");
  if (!on4(weights)) return set_error(APR_E_ALIGN, "weights are not 4-byte aligned");
  const size_t cb = code_bytes(w), sb = scale_bytes(w);
  const size_t wb = weights ? ((size_t)w.num_seqs * w.kv_heads * weights_ld) * 4 : 0;
  const Range outs[] = {{out, span_of(w.num_rows, ldo, width) * size, "out"}, {weights, wb, "weights"}};
  const Range ins[] = {{q, span_of(w.num_rows, ldq, width) * size, "q"},
                       {w.K, cb, "K"},
                       {w.V, cb, "V"},
                       {w.k_scale, sb, "k_scale"},
                       {w.v_scale, sb, "v_scale"},
                       {w.table, table_bytes(w), "page_table"},
                       {w.lens, (size_t)w.num_seqs * 4, "lens"},
                       {w.row_start, start_bytes(w), "row_start"}};
  rc = check_overlap(outs, ins);
  if (rc != APR_OK) return rc;
  rc = device_status_word(&w.status);
  if (rc != APR_OK) return rc;
  if (w.num_rows == 0) return launched(cudaMemsetAsync(weights, 0, wb, s), "attention");  // no row, no weight
  const Kv8Attention a{type,  q,       out,        ldq,       ldo, num_heads, scale > 0.f ? scale : 1.f / std::sqrt((float)w.dim),
                       weights, weights_ld, accumulate != 0,
                       rows->row_start && !rows->max_rows ? (w.num_rows + w.num_seqs - 1) / w.num_seqs : w.max_rows};
  const StreamOrder order(s);
  void* scratch = nullptr;
  rc = kv8_scratch(s, kv8_attention_scratch(w, a), &scratch);
  if (rc != APR_OK) return rc;
  return launched(launch_kv8_attention(w, a, scratch, s), "attention");
}

int run_prefill_attention(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, const void* q, long long ldq,
                          void* out, long long ldo, int num_heads, float scale, cudaStream_t s) {
  Kv8View w;
  int rc = view_of(cache, rows, true, false, &w);
  if (rc != APR_OK) return rc == 1 ? APR_OK : rc;
  rc = check_heads(w, type, q, ldq, out, ldo, num_heads, scale);
  if (rc != APR_OK) return rc;
  // what the segments cost is counted in 64 bits, for ranges of rows of any kind: of 128 pairs or more, each at most
  // (max_len + max_rows + a start) * group, and shares of six times the sum
  if ((long long)w.num_rows * num_heads > (1LL << 32) ||
      (double)w.num_seqs * ((double)w.max_rows * num_heads / 128. + num_heads) * ((double)w.max_len + w.max_rows + 4096.) *
              (num_heads / w.kv_heads) > 0x1p59)
    return set_error(APR_E_INVAL, "sizes beyond the supported limits");
  const size_t size = type_size(type), width = (size_t)num_heads * w.dim, cb = code_bytes(w), sb = scale_bytes(w);
  const Range outs[] = {{out, span_of(w.num_rows, ldo, width) * size, "out"}};
  const Range ins[] = {{q, span_of(w.num_rows, ldq, width) * size, "q"},
                       {w.K, cb, "K"},
                       {w.V, cb, "V"},
                       {w.k_scale, sb, "k_scale"},
                       {w.v_scale, sb, "v_scale"},
                       {w.table, table_bytes(w), "page_table"},
                       {w.lens, (size_t)w.num_seqs * 4, "lens"},
                       {w.row_start, start_bytes(w), "row_start"}};
  rc = check_overlap(outs, ins);
  if (rc != APR_OK) return rc;
  rc = device_status_word(&w.status);
  if (rc != APR_OK) return rc;
  const StreamOrder order(s);
  void* scratch = nullptr;
  rc = kv8_scratch(s, kv8_prefill_scratch(w), &scratch);
  if (rc != APR_OK) return rc;
  return launched(launch_kv8_prefill(w, type, q, ldq, out, ldo, num_heads, scale > 0.f ? scale : 1.f / std::sqrt((float)w.dim),
                                     scratch, s),
                  "prefill attention");
}

// ---------------------------------------------------------------- rotations
// Checks a rotation for `rows` rows of heads of `dim`, and fills the kernels' view of it.
int rope_view(const apr_rope* r, int dim, int rows, bool needs_positions, RopeView* w) {
  if (!r) return set_error(APR_E_INVAL, "null rope");
  if (r->rot_dim < 8 || r->rot_dim % 8 != 0 || r->rot_dim > dim)
    return failf(APR_E_INVAL, "rot_dim=%lld must be a multiple of 8 within the head's %lld dims", r->rot_dim, dim);
  if (r->num_positions < 1 || r->num_positions > (1 << 30))
    return failf(APR_E_INVAL, "num_positions=%lld must be within 1 and 2^30", r->num_positions);
  if (r->num_axes < 1 || r->num_axes > 16 || (r->num_axes > 1 && !r->pair_axis))
    return failf(APR_E_INVAL, "num_axes=%lld must be within 1 and 16, and 1 without pair_axis", r->num_axes);
  if (r->positions_ld != 0 && r->positions_ld < rows)
    return failf(APR_E_INVAL, "positions_ld=%lld is less than the call's %lld rows", r->positions_ld, rows);
  if (!r->table) return set_error(APR_E_INVAL, "null table");
  if (!r->positions && (needs_positions || r->num_axes > 1))
    return set_error(APR_E_INVAL, "null positions");
  if (!on16(r->table)) return set_error(APR_E_ALIGN, "the table is not 16-byte aligned");
  if (!on4(r->positions) || !on4(r->pair_axis))
    return set_error(APR_E_ALIGN, "positions or pair_axis are not 4-byte aligned");
  *w = RopeView{reinterpret_cast<const float2*>(r->table), r->pair_axis, r->positions, r->positions_ld ? r->positions_ld : rows,
                nullptr, r->num_positions, r->rot_dim / 2, r->num_axes, r->interleaved != 0};
  return APR_OK;
}
size_t rope_table_bytes(const RopeView& w) { return (size_t)w.num_positions * w.pairs * 8; }
size_t rope_positions_bytes(const RopeView& w, int rows) {
  return w.positions ? span_of(w.num_axes, w.positions_ld, rows) * 4 : 0;
}

// The rows x and out of heads that are rotated: sizes, alignment, and that out is x itself or does not meet it.
int check_rope_rows(int size, const void* x, long long ldx, const void* out, long long ldo, int rows, long long width,
                    const char* what) {
  if (ldx < width || ldo < width || ldx > (1LL << 28) || ldo > (1LL << 28))
    return failf(APR_E_INVAL, "row strides %lld and %lld must be within the rows' %lld elements and 2^28", ldx, ldo, width);
  if (!x || !out) return set_error(APR_E_INVAL, "null rows");
  if (!on16(x) || !on16(out) || ldx * size % 16 != 0 || ldo * size % 16 != 0)
    return failf(APR_E_ALIGN, "the rows (strides %lld, %lld) are not on 16-byte boundaries", ldx, ldo);
  if (!(x == out && (ldx == ldo || rows <= 1)) && rows_meet(x, ldx * size, width * size, out, ldo * size, width * size, rows))
    return set_error(APR_E_ALIAS, what);
  return APR_OK;
}
int check_norm(const float* norm, float eps) {
  if (!(eps >= 0.f) || !std::isfinite(eps)) return set_error(APR_E_INVAL, "eps must be finite and not negative");
  if (!on16(norm)) return set_error(APR_E_ALIGN, "the norm's weights are not 16-byte aligned");
  return APR_OK;
}

int run_rope_table(const float* inv_freq, int pairs, long long first, long long positions, double scale, float* table,
                   cudaStream_t s) {
  if (pairs < 1 || pairs > 256) return failf(APR_E_INVAL, "pairs=%lld must be within 1 and 256", pairs);
  if (first < 0 || positions < 0 || first > (1LL << 30) || positions > (1LL << 30) - first || positions * pairs > (1LL << 32))
    return failf(APR_E_INVAL, "positions %lld and %lld more are beyond 2^30, or 2^32 values", first, positions);
  // (what rounding took, 2^-48 of a value, is turned on with it: below 2^-100 it leaves float32's range)
  if (!(std::fabs(scale) <= 0x1p100) || (scale != 0. && std::fabs(scale) < 0x1p-100))
    return set_error(APR_E_INVAL, "scale must be 0 or of a magnitude within 2^-100 and 2^100");
  if (positions == 0) return APR_OK;
  if (!inv_freq || !table) return set_error(APR_E_INVAL, "null inv_freq or table");
  if (!on16(table) || !on4(inv_freq)) return set_error(APR_E_ALIGN, "the table is not 16-byte, or inv_freq not 4-byte aligned");
  if (meet(inv_freq, (size_t)pairs * 4, table, (size_t)positions * pairs * 8))
    return set_error(APR_E_ALIAS, "table overlaps inv_freq");
  unsigned* status;
  const int rc = device_status_word(&status);
  if (rc != APR_OK) return rc;
  return launched(launch_rope_table(inv_freq, pairs, first, positions, scale, table, s), "rope table");
}

int run_rope_rows(const apr_rope* rope, int type, const void* x, long long ldx, void* out, long long ldo, int num_rows,
                  int num_heads, int head_dim, const float* norm, float eps, cudaStream_t s) {
  const int size = type_size(type);
  if (!size) return failf(APR_E_INVAL, "unknown element type %lld", type);
  if (num_rows < 0 || num_rows > (1 << 24) || num_heads < 1 || num_heads > 65536 || (long long)num_rows * num_heads > (1LL << 32))
    return failf(APR_E_INVAL, "bad sizes: num_rows=%lld num_heads=%lld", num_rows, num_heads);
  if (head_dim < 8 || head_dim > 512 || head_dim % 8 != 0)
    return failf(APR_E_INVAL, "head_dim=%lld must be a multiple of 8 within 8 and 512", head_dim);
  RopeView w;
  if (num_rows == 0) return APR_OK;
  int rc = rope_view(rope, head_dim, num_rows, true, &w);
  if (rc != APR_OK) return rc;
  rc = check_norm(norm, eps);
  if (rc != APR_OK) return rc;
  const long long width = (long long)num_heads * head_dim;
  rc = check_rope_rows(size, x, ldx, out, ldo, num_rows, width, "out overlaps x without being it");
  if (rc != APR_OK) return rc;
  const Range outs[] = {{out, span_of(num_rows, ldo, width) * size, "out"}};
  const Range ins[] = {{w.table, rope_table_bytes(w), "table"},
                       {w.axis, w.axis ? (size_t)w.pairs : 0, "pair_axis"},
                       {w.positions, rope_positions_bytes(w, num_rows), "positions"},
                       {norm, norm ? (size_t)head_dim * 4 : 0, "norm"}};
  rc = check_overlap(outs, ins);
  if (rc != APR_OK) return rc;
  rc = device_status_word(&w.status);
  if (rc != APR_OK) return rc;
  return launched(launch_rope_rows(w, RopeRows{x, out, ldx, ldo, norm, eps, num_rows, num_heads, head_dim, 0}, type, s), "rope rows");
}

int run_rope_append(const apr_kv8_cache* cache, const apr_kv8_rows* rows, const apr_rope* rope, int type, const void* k,
                    const void* v, long long ld, const float* k_norm, const void* q, long long ldq, void* q_out,
                    long long ldqo, int num_heads, const float* q_norm, float eps, cudaStream_t s) {
  Kv8View w;
  int rc = view_of(cache, rows, true, false, &w);
  if (rc != APR_OK) return rc == 1 ? APR_OK : rc;
  rc = check_rows(w, type, k, v, ld);
  if (rc != APR_OK) return rc;
  RopeView r;
  rc = rope_view(rope, w.dim, w.num_rows, false, &r);
  if (rc != APR_OK) return rc;
  rc = check_norm(k_norm, eps);
  if (rc == APR_OK) rc = check_norm(q_norm, eps);
  if (rc != APR_OK) return rc;
  const size_t size = type_size(type), kv_width = (size_t)w.kv_heads * w.dim;
  if (!q != !q_out) return set_error(APR_E_INVAL, "q without q_out, or q_out without q");
  size_t q_width = 0;
  if (q) {
    if (num_heads < 1 || num_heads > 65536 || (long long)w.num_rows * num_heads > (1LL << 32))
      return failf(APR_E_INVAL, "bad num_heads=%lld", num_heads);
    q_width = (size_t)num_heads * w.dim;
    rc = check_rope_rows((int)size, q, ldq, q_out, ldqo, w.num_rows, (long long)q_width, "q_out overlaps q without being it");
    if (rc != APR_OK) return rc;
    for (const void* p : {k, v})
      if (rows_meet(q_out, ldqo * size, q_width * size, p, ld * size, kv_width * size, w.num_rows))
        return set_error(APR_E_ALIAS, "q_out overlaps k or v");
  }
  const size_t bytes = span_of(w.num_rows, ld, kv_width) * size, cb = code_bytes(w), sb = scale_bytes(w);
  const Range outs[] = {{w.K, cb, "K"}, {w.V, cb, "V"}, {w.k_scale, sb, "k_scale"}, {w.v_scale, sb, "v_scale"},
                        {q_out, q ? span_of(w.num_rows, ldqo, q_width) * size : 0, "q_out"}};
  const Range ins[] = {{w.table, table_bytes(w), "page_table"},
                       {w.lens, (size_t)w.num_seqs * 4, "lens"},
                       {w.row_start, start_bytes(w), "row_start"},
                       {r.table, rope_table_bytes(r), "table"},
                       {r.axis, r.axis ? (size_t)r.pairs : 0, "pair_axis"},
                       {r.positions, rope_positions_bytes(r, w.num_rows), "positions"},
                       {k_norm, k_norm ? (size_t)w.dim * 4 : 0, "k_norm"},
                       {q_norm, q_norm ? (size_t)w.dim * 4 : 0, "q_norm"}};
  rc = check_overlap(outs, ins);
  if (rc != APR_OK) return rc;
  for (const Range in : {Range{k, bytes, "k"}, Range{v, bytes, "v"}, Range{q, q ? span_of(w.num_rows, ldq, q_width) * size : 0, "q"}})
    for (int i = 0; i < 4; ++i) {  // (q_out has been looked at: rows that interleave)
      const Range one[] = {outs[i]}, in1[] = {in};
      rc = check_overlap(one, in1);
      if (rc != APR_OK) return rc;
    }
  rc = device_status_word(&w.status);
  if (rc != APR_OK) return rc;
  r.status = w.status;
  return launched(launch_rope_kv8_append(w, r, type, k, v, ld, k_norm, eps,
                                         RopeRows{q, q_out, ldq, ldqo, q_norm, eps, w.num_rows, q ? num_heads : 0, w.dim, 0}, s),
                  "rotating append");
}

int run_evict(const apr_kv8_cache* cache, const apr_kv8_rows* rows, const float* weights, long long weights_ld,
              int budget, int recent, const int* fresh_pages, int* table_out, int* lens_out, float* weights_out,
              long long weights_out_ld, int* kept, cudaStream_t s) {
  Kv8View w;
  int rc = view_of(cache, rows, false, true, &w);
  if (rc != APR_OK) return rc == 1 ? APR_OK : rc;
  if (budget < 1 || budget > (1 << 30) || recent < 0 || recent > budget)
    return failf(APR_E_INVAL, "budget=%lld must be positive, and recent=%lld within 0 .. budget", budget, recent);
  if (weights_ld < w.max_len || weights_ld > (1LL << 30) || weights_out_ld < budget || weights_out_ld > (1LL << 30))
    return failf(APR_E_INVAL, "weights_ld=%lld (>= max_len) or weights_out_ld=%lld (>= budget) is out of range",
                 weights_ld, weights_out_ld);
  if (!weights || !fresh_pages || (!table_out && w.table_ld > 0) || !lens_out || !weights_out || !kept)
    return set_error(APR_E_INVAL, "null pointer");
  for (const void* p : {(const void*)weights, (const void*)fresh_pages, (const void*)table_out, (const void*)lens_out,
                        (const void*)weights_out, (const void*)kept})
    if (!on4(p)) return set_error(APR_E_ALIGN, "an argument is not 4-byte aligned");
  const size_t bg = (size_t)w.num_seqs * w.kv_heads, page = (size_t)1 << w.page_shift;
  const size_t fresh = (budget + page - 1) / page;
  if (2 * fresh * w.kv_heads > 0x7fffffffull) return set_error(APR_E_INVAL, "sizes beyond the supported limits");
  const size_t cb = code_bytes(w), sb = scale_bytes(w);
  const Range outs[] = {{table_out, table_bytes(w), "table_out"},
                        {lens_out, (size_t)w.num_seqs * 4, "lens_out"},
                        {weights_out, bg * weights_out_ld * 4, "weights_out"},
                        {kept, bg * budget * 4, "kept"}};
  const Range ins[] = {{weights, bg * weights_ld * 4, "weights"},
                       {fresh_pages, (size_t)w.num_seqs * fresh * 4, "fresh_pages"},
                       {w.K, cb, "K"},
                       {w.V, cb, "V"},
                       {w.k_scale, sb, "k_scale"},
                       {w.v_scale, sb, "v_scale"},
                       {w.table, table_bytes(w), "page_table"},
                       {w.lens, (size_t)w.num_seqs * 4, "lens"}};
  rc = check_overlap(outs, ins);
  if (rc != APR_OK) return rc;
  rc = device_status_word(&w.status);
  if (rc != APR_OK) return rc;
  return launched(launch_kv8_evict(w, weights, weights_ld, budget, recent, fresh_pages, table_out, lens_out,
                                   weights_out, weights_out_ld, kept, s),
                  "evict");
}

// No exception leaves the C interface.
template <typename F>
int guarded(F f) {
  set_error(APR_OK, "");
  try {
    return f();
  } catch (const std::exception& e) {
    return set_error(APR_E_NOMEM, e.what());
  } catch (...) {
    return set_error(APR_E_NOMEM, "unknown exception");
  }
}

}  // namespace

extern "C" {

int apr_kv8_append(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, const void* k, const void* v,
                   long long ld, apr_stream_t stream) {
  return guarded([&] { return run_append(cache, rows, type, k, v, ld, (cudaStream_t)stream); });
}

int apr_kv8_read(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, void* k, void* v, long long ld,
                 apr_stream_t stream) {
  return guarded([&] { return run_read(cache, rows, type, k, v, ld, (cudaStream_t)stream); });
}

int apr_kv8_attention(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, const void* q, long long ldq,
                      void* out, long long ldo, int num_heads, float scale, float* weights, long long weights_ld,
                      int accumulate, apr_stream_t stream) {
  return guarded([&] {
    return run_attention(cache, rows, type, q, ldq, out, ldo, num_heads, scale, weights, weights_ld, accumulate,
                         (cudaStream_t)stream);
  });
}

int apr_kv8_prefill_attention(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, const void* q,
                              long long ldq, void* out, long long ldo, int num_heads, float scale,
                              apr_stream_t stream) {
  return guarded([&] {
    return run_prefill_attention(cache, rows, type, q, ldq, out, ldo, num_heads, scale, (cudaStream_t)stream);
  });
}

int apr_rope_table(const float* inv_freq, int pairs, long long first, long long positions, double scale, float* table,
                   apr_stream_t stream) {
  return guarded([&] { return run_rope_table(inv_freq, pairs, first, positions, scale, table, (cudaStream_t)stream); });
}

int apr_rope_rows(const apr_rope* rope, int type, const void* x, long long ldx, void* out, long long ldo, int num_rows,
                  int num_heads, int head_dim, const float* norm, float eps, apr_stream_t stream) {
  return guarded([&] {
    return run_rope_rows(rope, type, x, ldx, out, ldo, num_rows, num_heads, head_dim, norm, eps, (cudaStream_t)stream);
  });
}

int apr_rope_kv8_append(const apr_kv8_cache* cache, const apr_kv8_rows* rows, const apr_rope* rope, int type,
                        const void* k, const void* v, long long ld, const float* k_norm, const void* q, long long ldq,
                        void* q_out, long long ldqo, int num_heads, const float* q_norm, float eps,
                        apr_stream_t stream) {
  return guarded([&] {
    return run_rope_append(cache, rows, rope, type, k, v, ld, k_norm, q, ldq, q_out, ldqo, num_heads, q_norm, eps,
                           (cudaStream_t)stream);
  });
}

int apr_kv8_evict(const apr_kv8_cache* cache, const apr_kv8_rows* rows, const float* weights, long long weights_ld,
                  int budget, int recent, const int* fresh_pages, int* table_out, int* lens_out, float* weights_out,
                  long long weights_out_ld, int* kept, apr_stream_t stream) {
  return guarded([&] {
    return run_evict(cache, rows, weights, weights_ld, budget, recent, fresh_pages, table_out, lens_out, weights_out,
                     weights_out_ld, kept, (cudaStream_t)stream);
  });
}

}  // extern "C"
