/*
 * spec_logits.h - what stands between hidden states and the logits that a
 * verification reads, GB300: a 4-bit draft head (its quantisation and its
 * products with a few rows) and the per-request processing of logits.
 *
 * The conventions of spec_verify.h hold for every entry point here: device
 * pointers, row-major, caller-owned; nothing is allocated, freed or
 * synchronised; every call is asynchronous on `stream`; argument errors
 * return a negative spec_status before anything is launched; data errors set
 * bits in the optional `seq_error` / `*error_word`; the same inputs on the
 * same GPU give bit-identical outputs.
 */
#ifndef SPEC_LOGITS_H
#define SPEC_LOGITS_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* data-error bit of spec_process_logits, beside SPEC_ERR_TOKEN and
   SPEC_ERR_PARENT: a mask_index entry outside [-1, mask_rows)            */
#define SPEC_ERR_MASK 64

/* ---------------------------------------------------------------------- */
/* Per-request processing of logits: penalties for repeated tokens, biases */
/* and grammar masks, position by position.  Speculative sampling is       */
/* lossless for the distribution whose logits it is given (spec_verify.h): */
/* to sample a request's processed distribution, both the target and the   */
/* draft rows are processed, each row with the tokens before ITS position: */
/*  - chain (parent NULL): row i of sequence b follows b's history and the */
/*    drafted tokens [b, 0 .. i-1];                                        */
/*  - tree: row i is node i's; it follows the history and the tokens of    */
/*    the nodes on the path from the root to i, the root excluded (the     */
/*    root's token is the history's last).                                 */
/* One row alone, as drafting wants it, follows the history alone: append   */
/* the tokens drafted so far to it (and count them in history_len).         */
/* With s(v) = token v occurs in the history or on the path, and c(v) = its */
/* occurrences in the history from prompt_len[b] on and on the path:       */
/*    x1 = s ? (x > 0 ? x * (1 / repetition) : x * repetition) : x         */
/*    x2 = x1 - (frequency * c + (c > 0 ? presence : 0))                   */
/*    x3 = x2 + the sum of b's bias entries for v, in their order          */
/*    y  = allowed ? x3 : -inf                                             */
/* in float32, a rounding per operation (the penalty's product and sum are  */
/* one), rounded once more to the logits' type; an element that nothing    */
/* applies to keeps its bits, and -inf stays -inf.  A masked element is    */
/* -inf whatever it held (NaN included); a row whose mask allows nothing   */
/* is all -inf, which the verification reports as SPEC_ERR_NONFINITE.      */
/*  - `out` may be `logits` itself (with the same ld) or must not overlap  */
/*    it.                                                                  */
/*  - A history, drafted or bias token outside [0, V) and a history_len or */
/*    bias_len outside its range set SPEC_ERR_TOKEN: the token is ignored, */
/*    the length clamped.  A node whose parent is outside [0, i) sets      */
/*    SPEC_ERR_PARENT and counts as the root's child.  A mask_index        */
/*    outside [-1, mask_rows) sets SPEC_ERR_MASK: the row is not masked.   */
/*    Everything else of the sequence is processed all the same.           */
/*  - One kernel launch; two where many long histories over a large        */
/*    vocabulary are first gathered in the workspace.                      */
/* ---------------------------------------------------------------------- */
typedef struct spec_process_args {
  int B;                       /* sequences, 1..65535                              */
  int n;                       /* rows per sequence, 1..1024                       */
  int V;                       /* vocabulary size, 1..2,097,152                    */
  spec_dtype dtype;            /* of logits and out                                */
  long long ld;                /* row stride of logits (elements), >= V            */
  long long out_ld;            /* row stride of out, >= V                          */
  const void* logits;          /* [B, n] rows, 16-byte aligned base                */
  void* out;                   /* [B, n] rows, 16-byte aligned base                */
  const int* tokens;           /* [B, tokens_ld] drafted tokens (chain: the first  */
                               /* n - 1 are read) or node tokens (tree: entries    */
                               /* 1 .. n-1 are read); NULL: none (chain only)      */
  const int* parent;           /* [B, n] parent of each node, entry 0 not read;    */
                               /* NULL: a chain                                    */
  int tokens_ld;               /* >= n - 1 (chain), >= n (tree)                    */
  int history_ld;              /* tokens per history row, 0..268,435,456           */
  const int* history;          /* [B, history_ld] prompt and generated tokens, or  */
                               /* NULL: empty                                      */
  const int* history_len;      /* [B] tokens of each history, 0..history_ld (0 for */
                               /* a history of width 0, whose address may be NULL; */
                               /* not read without a history); NULL: history_ld    */
  const int* prompt_len;       /* [B] leading history tokens that are the prompt   */
                               /* (clamped to the history); NULL: 0                */
  const float* repetition;     /* [B], > 0; NULL: 1                                */
  const float* frequency;      /* [B]; NULL: 0                                     */
  const float* presence;       /* [B]; NULL: 0                                     */
  const int* bias_tokens;      /* [B, bias_ld], or NULL: no biases                 */
  const float* bias_values;    /* [B, bias_ld]                                     */
  const int* bias_len;         /* [B] entries of each list, 0..bias_ld (likewise); */
                               /* NULL: bias_ld                                    */
  int bias_ld;                 /* 0..268,435,456                                   */
  int mask_rows;               /* rows of mask, >= 1 when mask is given            */
  const unsigned* mask;        /* [mask_rows, mask_ld] words: bit v % 32 of word   */
                               /* v / 32 is 1 where v is allowed; NULL: no masks   */
  long long mask_ld;           /* words per mask row, >= ceil(V / 32)              */
  const int* mask_index;       /* [B, n] mask row of each row, -1: not masked;     */
                               /* NULL: row (b, i) uses mask row b * n + i         */
  int* seq_error;              /* out [B], optional                                */
  int* error_word;             /* in/out, optional: error bits OR-ed in            */
  void* workspace;             /* 256-byte aligned; needs no initialisation        */
  size_t workspace_bytes;
} spec_process_args;

/* history_ld and bias_ld as in the arguments (0 without a history, without   */
/* biases).  0 for sizes outside the limits.                                  */
size_t spec_process_workspace_size(int B, int n, int V, int history_ld, int bias_ld);
/* SPEC_EINVAL: a size outside the limits, a NULL required pointer, or out =  */
/* logits with another stride; SPEC_EDTYPE; SPEC_EALIGN: logits or out not    */
/* 16-byte aligned; SPEC_EWORKSPACE: workspace NULL, short or not 256-byte     */
/* aligned; SPEC_ECUDA: a launch failed.                                      */
spec_status spec_process_logits(const spec_process_args* args, cudaStream_t stream);

/* ---------------------------------------------------------------------- */
/* 4-bit weights with group scales.  A matrix [V, d] (an LM head: one row  */
/* per vocabulary entry) is held as                                        */
/*   codes  [V, codes_ld] bytes: code q(v, k), 0..15, in the low nibble of */
/*          byte k / 2 for even k, in the high nibble for odd k            */
/*   scales [d / group, scales_ld] bfloat16: s(g, v), one row per group    */
/*   zeros  [d / group, zeros_ld] bytes: z(g, v), 0..15; absent: 8         */
/* and stands for w(v, k) = s(k / group, v) * (q(v, k) - z(k / group, v)). */
/* group is 32, 64 or 128 and divides d.                                   */
/*                                                                         */
/* spec_quantize_int4 writes that form of a float32 or bfloat16 matrix,    */
/* every step in float32 with IEEE division and ties to even:              */
/*   without zeros  a = max |w| of the group, s = bf16(a / 7),             */
/*                  q = clamp(rint(w / s), -8, 7) + 8                      */
/*   with zeros     lo = min(0, min w), hi = max(0, max w),                */
/*                  s = bf16((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15), */
/*                  q = clamp(rint(w / s) + z, 0, 15)                      */
/*   s = 0          q = z (8 without zeros, z = 0 with): the weights are 0 */
/*   a group with a NaN or an infinity, or whose s overflows: s = NaN and  */
/*                  q = z likewise, so that products with it are NaN       */
/* One kernel launch.                                                      */
/* ---------------------------------------------------------------------- */
typedef struct spec_quantize_int4_args {
  int V;                       /* rows, 1..2,097,152                               */
  int d;                       /* columns, a multiple of group, 32..65536          */
  int group;                   /* 32, 64 or 128                                    */
  spec_dtype dtype;            /* of weights                                       */
  long long ld;                /* row stride of weights (elements), >= d           */
  long long codes_ld;          /* row stride of codes in bytes, >= d / 2, a        */
                               /* multiple of 16                                   */
  long long scales_ld;         /* row stride of scales (elements), >= V            */
  long long zeros_ld;          /* row stride of zeros (bytes), >= V, with zeros    */
  const void* weights;         /* [V, d], aligned to its element                   */
  void* codes;                 /* out, 16-byte aligned                             */
  void* scales;                /* out, 2-byte aligned                              */
  unsigned char* zeros;        /* out, or NULL: the form without zeros             */
} spec_quantize_int4_args;

/* SPEC_EINVAL, SPEC_EDTYPE, SPEC_EALIGN, SPEC_ECUDA as above.                */
spec_status spec_quantize_int4(const spec_quantize_int4_args* args, cudaStream_t stream);

/* ---------------------------------------------------------------------- */
/* Products of a few rows with a 4-bit matrix, e.g. the logits of the      */
/* tokens a draft model is about to draft:                                 */
/*   y(r, v) = sum_g s(g, v) * sum_{k in group g} (q(v, k) - z(g, v)) x(r, k) */
/* x bfloat16.  q - z is exact in bfloat16, the sums are float32 and the   */
/* scale multiplies a group's float32 sum, so no weight is rounded; y is   */
/* rounded once to its type.                                               */
/*  - Rows cost little until the products bound the call: up to 128 rows   */
/*    share one pass over the weights; more rows take further passes.      */
/*  - One kernel launch of at most one CTA per SM.  An entry whose width is */
/*    shared by several CTAs is summed in the order of the columns.        */
/*  - Nothing before a matrix's first entry or after its last one is read,  */
/*    wherever it starts; of what lies between rows (strides larger than    */
/*    the width) some bytes may be, and are not used.                       */
/*  - Workspace: its first 1024 bytes must be zero before its first use    */
/*    (and again after a call that reported SPEC_ERR_INTERNAL); a call     */
/*    leaves them zero, so calls that follow one another may share it.     */
/* ---------------------------------------------------------------------- */
typedef struct spec_int4_product_args {
  int R;                       /* rows, 1..65535                                   */
  int V;                       /* vocabulary size, 1..2,097,152                    */
  int d;                       /* width, a multiple of group, 32..65536            */
  int group;                   /* 32, 64 or 128                                    */
  spec_dtype out_dtype;        /* of out                                           */
  long long x_ld;              /* row stride of x (elements), >= d, a multiple of 8 */
  long long codes_ld;          /* as above                                         */
  long long scales_ld;
  long long zeros_ld;
  long long out_ld;            /* row stride of out (elements), >= V               */
  const void* x;               /* [R, d] bfloat16, 16-byte aligned                 */
  const void* codes;           /* 16-byte aligned                                  */
  const void* scales;          /* bfloat16                                         */
  const unsigned char* zeros;  /* or NULL                                          */
  void* out;                   /* out [R, out_ld], aligned to its element          */
  int* error_word;             /* in/out, optional: SPEC_ERR_INTERNAL when a       */
                               /* bounded wait gave up (never expected; out is     */
                               /* then not complete)                               */
  void* workspace;             /* 256-byte aligned                                 */
  size_t workspace_bytes;
} spec_int4_product_args;

/* 0 for sizes outside the limits above, and where                            */
/* ceil(R / 128) * ceil(V / 128) * ceil(d / 256) reaches 2^30.                */
size_t spec_int4_product_workspace_size(int R, int V, int d, int group);
/* SPEC_EINVAL (all sizes for which that is 0), SPEC_EDTYPE, SPEC_EALIGN,     */
/* SPEC_EWORKSPACE, SPEC_ECUDA.                                               */
spec_status spec_int4_product(const spec_int4_product_args* args, cudaStream_t stream);

/* Test hook for its bounded waits, as spec_verify.h has them for the          */
/* verifications.  While enabled, every stage of weights of the calls launched */
/* by this process waits for 16 bytes more than are copied, so its waits give  */
/* up after about 65 ms: *error_word gets SPEC_ERR_INTERNAL, out is not        */
/* written.  Nothing faults and nothing is left in flight.  Tests only: leave  */
/* it disabled (the default) in any other use.  SPEC_OK.                       */
spec_status spec_test_inject_product_copy_timeout(int enable);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LOGITS_H */
