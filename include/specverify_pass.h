/*
 * specverify_pass.h -- the verifier's pass: operators that a user of the
 * verification entry points (specverify.h) needs around the forward pass that
 * makes the target's rows, in each of its layers, and between two rounds.
 *
 *   sv_rope             rotary positions of a window's queries and keys
 *   sv_kv_write         its keys and values into a paged cache of 4 bits
 *   sv_kv_attention     attention of its nodes (a chain or a tree) over the
 *                       cache and over one another
 *   sv_kv_read          what the cache holds, in 16 or 32 bits
 *   sv_kv_commit        after verification: the cache keeps the accepted path
 *
 * A window holds the N nodes of one verification round: node 0 is the root
 * (the last token emitted, whose key is not cached yet), the others are the
 * drafts.  parent [B, N] is sv_verify_tree's array (parent[0] ignored,
 * 0 <= parent[i] < i); NULL means a chain (parent[i] = i - 1), as
 * sv_verify_chain verifies with gamma = N - 1.  With lens[b] tokens cached
 * before the window, node i's place in the cache is lens[b] + i and its
 * position lens[b] + depth(i).  A single token without drafts is a window of
 * one node.
 *
 * The conventions of specverify.h hold: device pointers owned by the caller,
 * the caller's workspace and stream, asynchronous calls that allocate nothing
 * and may be captured in a graph, argument checks on the host before anything
 * is enqueued, input errors found on the device as bits of the workspace's
 * error word.  Calls that overlap in time need a workspace each.  The same
 * call gives the same bits.
 *
 * Values are SV_BF16, SV_F16 or, where said, SV_F32.  Tensors [B, N, heads, D]
 * have a unit stride along D; `stride` points to 3 host values, the strides in
 * elements of sequence, node and head.  Strides are not negative and what is
 * written must not overlap itself; different heads of one tensor, of equal strides,
 * do not overlap.
 */
#ifndef SPECVERIFY_PASS_H
#define SPECVERIFY_PASS_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SV_F16 = 2 }; /* an sv_dtype of this header's entry points only */

typedef int32_t sv_pass_op;
enum {
  SV_PASS_ROPE = 0,
  SV_PASS_WRITE = 1,
  SV_PASS_READ = 2,
  SV_PASS_ATTENTION = 3,
  SV_PASS_COMMIT = 4
};

#define SV_MAX_HEADS 1024       /* query heads, key heads */
#define SV_MAX_PAGE_TOKENS (1 << 20)
#define SV_MAX_LAYERS 65536     /* layers of a commit */

/* Device error-word bits of these entry points: SV_DERR_TREE (a parent not
 * before its node, a path that does not rise) and SV_DERR_RANGE (a length, a
 * page or a count out of range; the same bit as in specverify_draft.h). */
#ifndef SV_DERR_RANGE
#define SV_DERR_RANGE 32
#endif

/*
 * A paged cache of one layer (or several of equal pages).  Tokens of sequence
 * b are numbered from 0; token t lies in page pages[b * max_pages +
 * t / page_tokens] at slot t % page_tokens.
 *
 * What a page holds: for each head D/2 + D/32 bytes a token of keys, as many
 * of values.  32 neighbouring values share a scale 2^(s - 127), s a byte; a
 * value is a code of 4 bits, sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (the
 * microscaling format MXFP4; the even-numbered value of a byte's two is in its
 * low half).  Per head, with P = page_tokens:
 *   keys           [P][D/2] bytes
 *   their scales   [P][D/32]
 *   values         [P/4][16][4][D/32]: a sixteenth of a row for 4 tokens
 *   their scales   [P/4][D/32][4]
 * Pages hold their heads one after another, page_stride bytes from page to
 * page (at least sv_kv_page_bytes), layers layer_stride bytes from one another.
 */
typedef struct sv_kv_cache {
  void* pool;            /* DEVICE, 16-byte aligned */
  const int32_t* pages;  /* DEVICE [B, max_pages] */
  int64_t page_stride;   /* bytes, a multiple of 16 */
  int64_t layer_stride;  /* bytes, a multiple of 16 (sv_kv_commit) */
  int32_t num_pages;     /* pages of the pool */
  int32_t max_pages;     /* pages a sequence can have */
  int32_t page_tokens;   /* a power of two, 16 .. SV_MAX_PAGE_TOKENS */
  int32_t H;             /* key heads */
  int32_t D;             /* 64, 128 or 256 */
  int32_t layers;        /* layers of the pool (sv_kv_commit) */
} sv_kv_cache;

/* Bytes of a page: H * page_tokens * (D + D / 16). */
sv_status sv_kv_page_bytes(int32_t H, int32_t D, int32_t page_tokens, int64_t* bytes);

/*
 * Workspace bytes for one call.  SV_PASS_ATTENTION reads all sizes; the others
 * take the fixed part only and read none.  SV_EINVAL / SV_EUNSUPPORTED for
 * shapes that the call would reject.
 */
sv_status sv_pass_workspace_size(sv_pass_op op, int32_t B, int32_t N, int32_t Hq, int32_t H, int32_t D,
                                 size_t* bytes);

/*
 * Rotary positions.  The first R values of each head are pairs (x_i, y_i),
 * i < R/2; at position t
 *   (x, y) -> factor * (x cos a - y sin a, y cos a + x sin a),  a = t * freq[i]
 * and with `inverse` the transposed map (a -> -a, the same factor): the
 * gradient.  What lies behind the first R values is copied.
 *   q [B, N, Hq, D], k [B, N, Hk, D] (Hk = 0: none), SV_BF16, SV_F16 or SV_F32
 *   freq [R/2] DEVICE double, angles a position (sv_rope_frequencies);
 *     2 <= R <= D, R even, any D up to 8192
 *   interleaved: pairs are (2i, 2i+1), else (i, i + R/2)
 *   positions [B, N] int32; or NULL: lens[b] (NULL: 0) + depth of the node in
 *     parent [B, N] (NULL: its number); with parent, N <= SV_MAX_N
 * out_q, out_k may be q, k (the same pointer and strides: in place) and must
 * not overlap them otherwise; all may be views of different heads of one tensor
 * (a fused projection), with equal strides.  Angles are formed in 64 bits and
 * reduced to a turn, so far positions keep their digits; sine, cosine and products
 * are of 32 bits (off by 2^-21 of |x| + |y| at most).  A node whose parent is not
 * before it sets SV_DERR_TREE and has depth 0.  All N nodes turn, padding too.
 */
sv_status sv_rope(const void* q, const int64_t* q_stride, const void* k, const int64_t* k_stride, sv_dtype dt,
                  int32_t B, int32_t N, int32_t Hq, int32_t Hk, int32_t D, int32_t R, const double* freq, float factor,
                  int32_t interleaved, int32_t inverse, const int32_t* positions, const int32_t* lens,
                  const int32_t* parent, void* out_q, const int64_t* out_q_stride, void* out_k,
                  const int64_t* out_k_stride, void* ws, size_t ws_bytes, void* stream);

typedef int32_t sv_rope_kind;
enum {
  SV_ROPE_PLAIN = 0,   /* theta^(-2i/R) */
  SV_ROPE_LINEAR = 1,  /* divided by `scale`: positions interpolated */
  SV_ROPE_BASE = 2,    /* theta * scale^(R/(R-2)) in theta's place */
  SV_ROPE_PARTS = 3    /* angles of more than `fast` turns over `original` positions stay, those of less than `slow` are
                          divided by `scale`, in between a ramp over i; out_factor = 0.1 ln(scale) + 1 */
};

/*
 * Host helper: the angles a position of R/2 pairs into the HOST array
 * out_freq, and the factor on what is rotated (1 but for SV_ROPE_PARTS) into
 * *out_factor.  scale >= 1; original, fast and slow (> 0, fast > slow) are read
 * by SV_ROPE_PARTS only.
 */
sv_status sv_rope_frequencies(sv_rope_kind kind, int32_t R, double theta, double scale, int32_t original, double fast,
                              double slow, double* out_freq, float* out_factor);

/*
 * Keys and values of a window (or a prompt) into the cache: token n of
 * sequence b goes to place lens[b] + n, for n < news[b] (NULL: N).
 *   k, v [B, N, H, D], SV_BF16, SV_F16 or SV_F32; 16-byte aligned rows
 *   lens [B], news [B] int32
 * A block of 32 values whose largest magnitude a lies in [2^e, 2^(e+1)) is
 * held at scale 2^(e-2), from 1.75 * 2^e on at 2^(e-1) (scales are kept in
 * [2^-126, 2^125]): each value becomes the nearest that the codes give, ties
 * to the even code, off by at most one scale (a / 4 or less).  A block with a
 * NaN or an infinity reads back as NaN.
 * A length or count out of range (lens < 0, news outside [0, N], lens + news
 * beyond the table) sets SV_DERR_RANGE and leaves the whole sequence as it
 * was; a page outside [0, num_pages) does so for its tokens.  Pages that
 * several sequences share are for reading: what two tokens of a call write to
 * one place is undefined.
 */
sv_status sv_kv_write(const void* k, const int64_t* k_stride, const void* v, const int64_t* v_stride, sv_dtype dt,
                      const sv_kv_cache* cache, const int32_t* lens, const int32_t* news, int32_t B, int32_t N,
                      void* ws, size_t ws_bytes, void* stream);

/*
 * What the cache holds: tokens start[b] .. start[b] + count[b] - 1 into rows 0
 * .. count[b] - 1 of out_k, out_v [B, N, H, D] (SV_BF16, SV_F16 or SV_F32,
 * 16-byte aligned rows); the rows behind are left as they were.  start NULL: 0;
 * count NULL: N.  bf16 holds every value exactly, fp16 where it lies in
 * its range.  Errors as at sv_kv_write; the rows concerned are left as they
 * were.
 */
sv_status sv_kv_read(const sv_kv_cache* cache, const int32_t* start, const int32_t* count, int32_t B, int32_t N,
                     sv_dtype dt, void* out_k, const int64_t* k_stride, void* out_v, const int64_t* v_stride,
                     void* ws, size_t ws_bytes, void* stream);

/*
 * Attention of a window's nodes over the cache, whose window has been written.
 * With d = position(i) - position(j), head h of the Hq query heads reading key
 * head h / (Hq / H), token j before the window or i itself or one of its
 * ancestors, and d < reach where reach > 0:
 *   s_ij = scale * q_i . k_j;  cap > 0: s = cap * tanh(s / cap);
 *   slopes: s = s - slopes[h] * d
 *   out_i = sum_j softmax_j(s_i) v_j,  out_lse_i = log sum_j exp(s_ij)
 *   q, out [B, N, Hq, D], SV_BF16 or SV_F16, 16-byte aligned rows; out must
 *     not overlap q
 *   lens [B], news [B] (NULL: N) int32: nodes news[b] .. N - 1 are padding,
 *     their outputs are left as they were
 *   parent [B, N] or NULL (a chain); N <= SV_MAX_N
 *   scale, cap finite, below 2^127 in magnitude
 *   slopes [Hq] float or NULL; out_lse [B, N, Hq] float or NULL, apart from
 *     q and out
 * Hq is a multiple of cache->H.  A sequence whose length or count is out of
 * range sets SV_DERR_RANGE and is left as it was.  A page outside [0,
 * num_pages) that has a token which the root sees, or one behind it, sets it too;
 * such a page's tokens count as masked (what lies wholly before the reach may be
 * gone).  A row that sees nothing is 0, its out_lse -inf.  A node whose parent is
 * not before it sets SV_DERR_TREE and sees the tokens before the window and itself.
 * NaN in a token that a row does not see does not reach it; queries are finite (a
 * row with a NaN or an infinity is NaN).
 *
 * The cache is read once for all query heads of a key head and up to 256 rows
 * (192 at D = 128, 64 at D = 256) of nodes x heads.  Keys become bf16 as they are
 * multiplied, which holds them exactly, and are multiplied by the queries (fp16:
 * by two parts of bf16 whose sum a query is).  Products, sums and the softmax are
 * held in 32 bits (a cap is off by 2^-21 of itself); probabilities are rounded to
 * the 8 bits of bf16 (fp16: 16 bits) before they multiply the values, and are
 * summed as rounded: a result is off by up to 2^-8 (2^-16) of how far the values
 * that it averages lie from it, beside the rounding of its own type.
 */
sv_status sv_kv_attention(const void* q, const int64_t* q_stride, sv_dtype dt, const sv_kv_cache* cache,
                          const int32_t* lens, const int32_t* news, const int32_t* parent, int32_t B, int32_t N,
                          int32_t Hq, float scale, float cap, const float* slopes, int32_t reach, void* out,
                          const int64_t* out_stride, float* out_lse, void* ws, size_t ws_bytes, void* stream);

/*
 * The cache after a verification: of each window the root and the accepted
 * path stay, in all of the pool's layers.  For j < n[b] the token at place
 * lens[b] + path[b, j] moves to lens[b] + 1 + j, and
 *   out_lens[b] = lens[b] + 1 + n[b].
 *   n [B], path [B, M]: out_len and out_path of sv_verify_tree (M its
 *     max_depth; what stands behind n[b] is not read); path NULL: a chain
 *     (out_n of sv_verify_chain), nothing moves
 *   out_lens [B] must not overlap lens, n or path
 * n[b] = -1 leaves a sequence as it was (it took no part), out_lens[b] =
 * lens[b].  So does a path that does not rise from 1 on within SV_MAX_N nodes,
 * which sets SV_DERR_TREE, and n outside [-1, M] (a chain: n < -1), a length out
 * of range or a page outside [0, num_pages) that a token moves from or to, which
 * sets SV_DERR_RANGE.  0 <= M <= SV_MAX_N; a path of M = 0 (any pointer but NULL,
 * not read) lets the root alone stay.
 */
sv_status sv_kv_commit(const sv_kv_cache* cache, const int32_t* lens, const int32_t* n, const int32_t* path, int32_t B,
                       int32_t M, int32_t* out_lens, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_PASS_H */
