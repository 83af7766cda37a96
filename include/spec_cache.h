/*
 * spec_cache.h - the key-value cache that a verification's target rows come
 * from, GB300: heads rotated by their positions, keys and values appended to
 * a paged cache of 8-bit codes, and the attention of drafted rows (a chain's
 * or a tree's) over that cache.
 *
 * Staged Speculative Decoding (arXiv 2308.04623), abstract: the speculative
 * batch is a tree, so a drafted row attends to the committed tokens and to
 * the nodes on its own root path.  PipeSpec review, "What carries the
 * argument": a buffer keeps the verified prefix and is rolled back to the
 * last verified token: here by its length alone (chains), or by appending the
 * kept path's rows once more (trees).
 *
 * The conventions of spec_verify.h hold for every entry point: device
 * pointers, caller-owned; nothing is allocated, freed or synchronised; every
 * call is asynchronous on `stream`; argument errors return a negative
 * spec_status before anything is launched; the same inputs on the same GPU
 * give bit-identical outputs.  One difference: data-error bits are OR-ed into
 * `seq_error` as well as into `*error_word` (the caller zeroes both).
 *
 * The cache.  Tokens lie in pages of `page` tokens (16, 32, 64 or 128);
 * entry t / page of a sequence's row of the block table names the page that
 * holds its token t, at place t % page.  Keys and values are each held as
 *   codes [pages, H, page, D] bytes, e4m3 (4-bit exponent, 3-bit mantissa,
 *         no infinities, 0x7f and 0xff NaN), and
 *   exps  [pages, H] signed bytes, -100..100: one exponent per page and head;
 * code c of page p and head h stands for c * 2^exps[p, h].
 */
#ifndef SPEC_CACHE_H
#define SPEC_CACHE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* data-error bits beside those of spec_verify.h                            */
#define SPEC_ERR_CACHE 128    /* a page, a length or a count of rows outside its range */
#define SPEC_ERR_POSITION 256 /* a position outside the rotation table                 */

/* ---------------------------------------------------------------------- */
/* Rotary positions.  A rotation table [rows, rot] float32 holds for each  */
/* position t the cosines, then the sines of t * freq[i], i < rot / 2,     */
/* times a magnitude (angles and functions in 64 bits, rounded once).      */
/* Long contexts are a matter of freq and magnitude.                       */
/* ---------------------------------------------------------------------- */
/* rows 1..2^30, rot even, 2..1024; freq [rot / 2] doubles on the device.   */
/* SPEC_EINVAL, SPEC_EALIGN (freq or table not aligned to its element),    */
/* SPEC_ECUDA.                                                             */
spec_status spec_rotation_table(int rows, int rot, const double* freq, double magnitude, float* table,
                                cudaStream_t stream);

/* The first rot elements of every head are rotated, pair i = (a, b) by row */
/* t of the table, t the row's position:                                    */
/*    a' = a cos - b sin,  b' = b cos + a sin                               */
/* pairs = 0: a and b are elements i and i + rot / 2; pairs = 1: elements   */
/* 2 i and 2 i + 1.  The others are copied.  transpose = 1: the sines are   */
/* negated, which is the inverse rotation (times the magnitude squared) and */
/* the gradient: d x = the transposed rotation of d out.  In float32, a     */
/* rounding per operation (two products, one sum), rounded to the type.     */
/*  - out may be x itself (with the same strides) or must not overlap it.   */
/*  - A position outside [0, table_rows) sets SPEC_ERR_POSITION; the row's   */
/*    rotated elements are NaN.                                             */
/*  - One kernel launch.                                                    */
typedef struct spec_rotate_args {
  int B;                       /* sequences, 1..65535                              */
  int n;                       /* rows per sequence, 1..2^20                       */
  int H;                       /* heads per row, 1..1024                           */
  int D;                       /* elements per head, even, 2..1024                 */
  int rot;                     /* rotated elements per head, even, 2..D            */
  int pairs;                   /* 0 or 1                                           */
  int transpose;               /* 0 or 1                                           */
  spec_dtype dtype;            /* of x and out                                     */
  long long x_ld[3];           /* strides of x in elements: sequence, row, head    */
  long long out_ld[3];         /* strides of out                                   */
  const void* x;               /* [B, n, H, D], unit element stride, aligned to    */
  void* out;                   /* out: its element                                 */
  const float* table;          /* [table_rows, rot], 16-byte aligned               */
  int table_rows;              /* >= 1                                             */
  const int* positions;        /* [B, n]; NULL: prefix_len[b] + i                  */
  const int* prefix_len;       /* [B]; NULL: 0 (not read with positions)           */
  int* seq_error;              /* in/out [B], optional: error bits OR-ed in        */
  int* error_word;             /* in/out, optional                                 */
} spec_rotate_args;

/* SPEC_EINVAL: a size outside its limits or a NULL required pointer;        */
/* SPEC_EDTYPE; SPEC_EALIGN; SPEC_ECUDA.                                     */
spec_status spec_rotate_heads(const spec_rotate_args* args, cudaStream_t stream);

/* ---------------------------------------------------------------------- */
/* Appending rows to the cache, keys rotated on the way.  Row i of sequence */
/* b's rows goes to token prefix_len[b] + i:                                */
/*  - without a path, its rows are k[b, 0 .. count[b]);                     */
/*  - with a path (spec_verify_tree's path_nodes and path_len, the root     */
/*    counted), they are k[b, path_nodes[b][0 .. path_len[b]]]: the kept    */
/*    nodes' rows, written over what was appended for the whole tree.        */
/* Of each page and head that gets rows, with a the largest finite |x| of   */
/* those rows (of keys before their rotation):                              */
/*    e = ceil(log2 a) - 7, within [-100, 100] (a = 0: -100), and not below  */
/*        the page's exponent where it holds tokens before prefix_len[b]     */
/*    code = e4m3(y * 2^-e), y = x or the rotated x in float32 (a rounding   */
/*        per operation), to nearest, ties to even                          */
/* so codes of rows that are appended stay within 128 (keys within 128      */
/* sqrt 2 times the table's magnitude), 13 binades above the least normal   */
/* code.  Where e grows, the page's tokens before prefix_len[b] are scaled   */
/* along (exact but for codes that become subnormal).  Nothing else of the  */
/* cache changes.                                                           */
/*  - No two entries of the block table that get rows, of one sequence or of */
/*    two, may name the same page.                                           */
/*  - A NaN, an infinity or a y beyond 448 * 2^e becomes a NaN code and sets */
/*    SPEC_ERR_NONFINITE.                                                   */
/*  - A position outside the table sets SPEC_ERR_POSITION: the key's rotated */
/*    elements become NaN codes.                                            */
/*  - A prefix_len < 0, a count outside [0, n], a path_len outside           */
/*    [0, max_depth] or rows past the block table set SPEC_ERR_CACHE, a path */
/*    node outside [0, n) SPEC_ERR_PARENT: the sequence is skipped.  A page  */
/*    outside [0, pages) sets SPEC_ERR_CACHE: its rows are not written.  A   */
/*    sequence whose path_nodes[b][0] is -1 is skipped without a bit.        */
/*  - One kernel launch.                                                    */
/* ---------------------------------------------------------------------- */
typedef struct spec_append_args {
  int B;                       /* sequences, 1..65535                              */
  int n;                       /* rows of k and v per sequence, 1..2^20            */
  int H;                       /* key-value heads, 1..1024                         */
  int D;                       /* elements per head, a multiple of 16, 16..256     */
  int page;                    /* tokens per page: 16, 32, 64 or 128               */
  int pages;                   /* pages of the cache, >= 1; pages * H * page <= 2^31 - 1 */
  int table_pages;             /* entries per block-table row, >= 1; times page <= 2^30 */
  int rot;                     /* rotated elements per key head, even, 0..D; 0: none */
  int pairs;                   /* as spec_rotate_args has it                       */
  int table_rows;              /* with rot                                         */
  int max_depth;               /* path_nodes has max_depth + 1 columns, 0..65534   */
  spec_dtype dtype;            /* of k and v                                       */
  long long k_ld[3];           /* strides in elements: sequence, row, head         */
  long long v_ld[3];
  const void* k;               /* [B, n, H, D], aligned to its element             */
  const void* v;
  const float* table;          /* [table_rows, rot], 16-byte aligned; with rot     */
  const int* positions;        /* [B, n] position of each row of k; NULL: the      */
                               /* token it goes to                                 */
  const int* prefix_len;       /* [B] tokens before the appended ones; NULL: 0     */
  const int* count;            /* [B] rows of each sequence (no path); NULL: n     */
  const int* path_nodes;       /* [B, max_depth + 1], or NULL: no path             */
  const int* path_len;         /* [B], with path_nodes                             */
  const int* block_table;      /* [B, table_pages]                                 */
  void* k_codes;               /* in/out, 16-byte aligned                          */
  void* v_codes;
  signed char* k_exps;         /* in/out                                           */
  signed char* v_exps;
  int* seq_error;              /* in/out [B], optional                             */
  int* error_word;             /* in/out, optional                                 */
} spec_append_args;

/* SPEC_EINVAL, SPEC_EDTYPE, SPEC_EALIGN, SPEC_ECUDA as above.               */
spec_status spec_append_cache(const spec_append_args* args, cudaStream_t stream);

/* ---------------------------------------------------------------------- */
/* Attention of drafted rows over the cache.  Sequence b's tokens are the   */
/* prefix_len[b] committed ones and the count[b] drafted ones after them,   */
/* all appended before.  Row i, i < count[b], of query head h reads head    */
/* h / (Hq / H) of the cache at the tokens                                  */
/*   t < prefix_len[b], and t = prefix_len[b] + j for                       */
/*   chain (parent NULL): j <= i;                                           */
/*   tree: j = i and every ancestor j of node i                             */
/* and gives  out = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale * q . k_t).  */
/* q bfloat16, out bfloat16.  Scores, maxima, weights, their sums and the   */
/* output's sums are float32; a query enters the products as the sum of two */
/* e4m3 numbers relative to its own largest element (exact to 2^-18 of that */
/* element), a weight times its page's 2^exponent as the sum of two relative */
/* to the largest of up to 256 tokens around it (to 2^-8 of itself, or 2^-18 */
/* of that largest), codes as they are.                                     */
/*  - Rows i >= count[b] get zeros.                                         */
/*  - A NaN code, or a NaN or infinite query element, makes NaN of the rows  */
/*    that read it (a value's NaN of its element of them at least), and of  */
/*    no others.  Codes behind a sequence's last token are not used,        */
/*    whatever they hold.                                                   */
/*  - A prefix_len < 0, a count outside [0, n] or tokens past the block     */
/*    table set SPEC_ERR_CACHE: the sequence's rows are zeros.  A page       */
/*    outside [0, pages) sets SPEC_ERR_CACHE: the rows that read it are NaN. */
/*    A parent outside [0, i) sets SPEC_ERR_PARENT: the node counts as the  */
/*    root's child.  A bounded wait that gives up sets SPEC_ERR_INTERNAL     */
/*    (never expected; the call's out is then not complete).                */
/*  - Two kernel launches: the rows' parts and their joining.               */
/*  - The workspace needs no initialisation and nothing in it outlives a    */
/*    call; two calls that can run at the same time need two.               */
/* ---------------------------------------------------------------------- */
typedef struct spec_attend_args {
  int B;                       /* sequences, 1..65535                              */
  int n;                       /* rows per sequence, 1..1024                       */
  int Hq;                      /* query heads, a multiple of H, up to 1024         */
  int H;                       /* key-value heads, 1..1024                         */
  int D;                       /* elements per head, a multiple of 16, 16..256     */
  int page;                    /* as in spec_append_args                           */
  int pages;
  int table_pages;
  float scale;                 /* of the scores, finite and > 0                    */
  long long q_ld[3];           /* strides in elements (sequence, row, head),       */
                               /* multiples of 8                                   */
  long long out_ld[3];         /* strides of out                                   */
  const void* q;               /* [B, n, Hq, D] bfloat16, 16-byte aligned          */
  void* out;                   /* out [B, n, Hq, D] bfloat16                       */
  const int* prefix_len;       /* [B]; NULL: 0                                     */
  const int* count;            /* [B] drafted rows, 0..n; NULL: n                  */
  const int* parent;           /* [B, n], entry 0 not read; NULL: a chain          */
  const int* block_table;      /* [B, table_pages]                                 */
  const void* k_codes;         /* 16-byte aligned                                  */
  const void* v_codes;
  const signed char* k_exps;
  const signed char* v_exps;
  int* seq_error;              /* in/out [B], optional                             */
  int* error_word;             /* in/out, optional                                 */
  void* workspace;             /* 256-byte aligned                                 */
  size_t workspace_bytes;
} spec_attend_args;

/* 0 for sizes outside the limits.                                           */
size_t spec_attend_workspace_size(int B, int n, int Hq, int H, int D);
/* SPEC_EINVAL (also where B * H * ceil(n * Hq / H / 16) * (table_pages *     */
/* page / 128 + 1) could reach 2^31), SPEC_EALIGN, SPEC_EWORKSPACE, SPEC_ECUDA */
/* as above.                                                                 */
spec_status spec_attend_cache(const spec_attend_args* args, cudaStream_t stream);

/* Test hook for its bounded waits, as spec_verify.h has them for the          */
/* verifications.  While enabled, every tile of codes of the calls launched by */
/* this process waits for 16 bytes more than are copied, so its waits give up   */
/* after about 65 ms: *error_word gets SPEC_ERR_INTERNAL.  Nothing faults and  */
/* nothing is left in flight.  Tests only.  SPEC_OK.                           */
spec_status spec_test_inject_cache_copy_timeout(int enable);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H */
