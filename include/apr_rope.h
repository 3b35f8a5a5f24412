/*
 * apr_rope.h — C ABI of the rotations by position (GB300, sm_103a): what lies
 * between a chunk's qkv projection and its attention. Part of libapr_qgemm;
 * errors, streams and apr_stream_status are those of apr_qgemm.h, the
 * 8-bit cache and its rows those of apr_kv8.h.
 *
 *   apr_rope_table       cosines and sines of positions times frequencies
 *   apr_rope_rows        rotates rows of heads, behind an optional norm of each head
 *   apr_rope_kv8_append  apr_rope_rows of k on its way into the 8-bit cache
 *                        (apr_kv8_append), with the q rows rotated beside it
 *
 * A rotation. Pair i of a head, i < rot_dim / 2, is its dims (i, i + rot_dim /
 * 2), or with `interleaved` (2 i, 2 i + 1). A row's position on the axis a =
 * pair_axis[i] (0 without pair_axis) says which row of the table turns it: with
 * (c, s) = table[positions[a][row]][i] and the pair's values (x, y)
 *   x' = f32(f32(x c) - f32(y s)),   y' = f32(f32(y c) + f32(x s)),
 * rounded to the rows' type. Dims past rot_dim pass. One axis is the usual
 * rotation; several are those of images and video (time, height, width), with
 * the pairs of each axis in any order: blocks, or neighbours in turn. What
 * stretches a context (scaled or divided frequencies, a factor on cosines and
 * sines) is in the table.
 *
 * With a norm (a weight for each dim of a head) the values are first
 *   f32(f32(x r) * weight),   r = f32(1 / sqrt(mean of x^2 over the head + eps)),
 * the mean and root to more than 40 bits, whatever the values' magnitude and
 * eps (r itself has float32's range: a head of a root mean square of 2^126 or less. A
 * head with a NaN or an infinity in it, or of zeros without an eps, becomes NaN). So
 * the result is the same on every path, whatever order a sum is taken in, but for
 * one r in some 10^5. Heads of a mean and eps beyond 2^+-100 take longer.
 *
 * Positions and axes are device arrays, read when the kernels run: an axis not
 * below num_axes counts as axis 0, a position that the table does not have as
 * position 0, and each sets a bit of the device status word (the next
 * apr_stream_status returns APR_E_INVAL; the call's outputs are then
 * unspecified). All pointers are device pointers, caller owned. Calls are asynchronous on
 * the stream, may be captured, take no scratch, and touch none of their arguments
 * before the work ahead of them is done.
 */
#ifndef APR_ROPE_H
#define APR_ROPE_H

#include "apr_kv8.h"
#include "apr_qgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct apr_rope {
  const float* table;             /* [num_positions][rot_dim / 2][2], on a 16-byte boundary */
  int num_positions;              /* 1 .. 2^30 */
  int rot_dim;                    /* a multiple of 8, at most the head's dim */
  int interleaved;                /* 0: pair i is dims i and i + rot_dim / 2; else 2 i and 2 i + 1 */
  const unsigned char* pair_axis; /* [rot_dim / 2], on a 4-byte boundary, or NULL */
  int num_axes;                   /* 1 .. 16 (1 without pair_axis) */
  const int* positions;           /* [num_axes][positions_ld] */
  int positions_ld;               /* 0: the rows of the call; else at least as many */
} apr_rope;

/*
 * table[p][i] = f32(scale cos(a)), f32(scale sin(a)), a = (first + p) inv_freq[i]
 * exactly, for 0 <= p < positions, 0 <= i < pairs: within half a step of float32 and 2^-40 (times
 * scale). Angles of far positions lose nothing.
 *   inv_freq  [pairs] float32, magnitudes up to 2^10; pairs 1 .. 256
 *   first     >= 0, first + positions <= 2^30; positions * pairs <= 2^32
 *   scale     0, or magnitudes of 2^-100 to 2^100 (the factor that some stretched rotations have; 1 otherwise)
 * positions == 0 is a no-op.
 */
int apr_rope_table(const float* inv_freq, int pairs, long long first, long long positions, double scale,
                   float* table, apr_stream_t stream);

/*
 * out = the rotated (and normed) rows x.
 *   rope      positions must be given
 *   x, out    [num_rows][ldx], [num_rows][ldo] rows of num_heads * head_dim elements
 *             of `type` (APR_T_F32, APR_T_F16, APR_T_BF16), rows on 16-byte
 *             boundaries; out may be x itself (with ldo == ldx), and may
 *             interleave with it as another slice of the same wider rows
 *   head_dim  a multiple of 8, 8 .. 512;  num_heads 1 .. 65536, num_rows 0 .. 2^24
 *   norm      [head_dim] float32 on a 16-byte boundary, or NULL;  eps >= 0 and finite
 */
int apr_rope_rows(const apr_rope* rope, int type, const void* x, long long ldx, void* out, long long ldo, int num_rows,
                  int num_heads, int head_dim, const float* norm, float eps, apr_stream_t stream);

/*
 * The same bits as apr_rope_rows of k and q, then apr_kv8_append of the rotated
 * k and of v, in one launch.
 *   cache, rows, type, k, v, ld   as for apr_kv8_append
 *   rope      positions == NULL: a row's position in its sequence, on the one
 *             axis (0 for rows before a sequence's start)
 *   k_norm    as norm above, of the head_dim dims of k's heads, or NULL
 *   q, q_out  [num_rows][ldq], [num_rows][ldqo] rows of num_heads * head_dim
 *             elements of `type`, or both NULL; q_out may be q itself (with
 *             ldqo == ldq) and may interleave with q, k and v as another slice of
 *             the same rows
 *   q_norm    of q's heads, or NULL;  eps is that of both norms
 * q rows of no sequence (ahead of row_start[0], or from row_start[num_seqs] on)
 * are left alone, and so are their positions.
 */
int apr_rope_kv8_append(const apr_kv8_cache* cache, const apr_kv8_rows* rows, const apr_rope* rope, int type,
                        const void* k, const void* v, long long ld, const float* k_norm, const void* q, long long ldq,
                        void* q_out, long long ldqo, int num_heads, const float* q_norm, float eps,
                        apr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* APR_ROPE_H */
