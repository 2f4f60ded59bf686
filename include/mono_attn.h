/*
 * mono_attn — the attention half's decode operators beside the FFN half-layer
 * of mono_ffn.h, on NVIDIA B200 (sm_100a).  Between them they make the
 * y_attn that mono_ffn_step_pending takes:
 *
 *   mono_proj    y = x W^T for 1-8 rows, W in 4 bits with group scales
 *                (the q, k, v and output projections, an output head)
 *   mono_rope    rotary positions on q (or k)
 *   mono_attn_append  new keys and values into a paged 8-bit cache, the keys
 *                rotated on the way
 *   mono_attn_attend  attention of the new tokens over that cache
 *
 * Conventions for every entry point (as in mono_ffn.h):
 *   - Return 0 on success or a negative MONO_ERR_* code; mono_attn_last_error
 *     then holds every reason, newline-separated.  Nothing is thrown.
 *   - Device pointers are CUDA device addresses on the plan's device (for
 *     mono_rope_apply: the current device); the caller keeps ownership.
 *   - `stream` is a cudaStream_t of that device (NULL = the legacy default
 *     stream).  Calls are asynchronous, allocate nothing and do not
 *     synchronise the host unless stated; all may be captured in a graph.
 *   - Nothing traps on the device, and no wait spins on another CTA.
 *   - Strides count elements; the innermost dimension is contiguous.
 */
#ifndef MONO_ATTN_H
#define MONO_ATTN_H

#include "mono_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a value in lens, n_new or the page table that a kernel could not use (mono_attn_query_error) */
#define MONO_ERR_BAD_INDEX (-9)

/* ------------------------------------------------------ rotary positions */

enum {
  MONO_ROPE_NONE = 0,   /* theta^(-2i/rot_dim) radians a position */
  MONO_ROPE_LINEAR = 1, /* positions divided by factor */
  MONO_ROPE_NTK = 2,    /* theta times factor^(rot_dim / (rot_dim - 2)) */
  MONO_ROPE_YARN = 3    /* the interpolated and the plain frequency blended by a ramp over the pairs (YaRN) */
};

typedef struct {
  int rot_dim;       /* rotated dimensions of a head, even, 2..256 */
  int offset;        /* the first of them, even (0: the head's start; head_dim - rot_dim: its end) */
  int interleaved;   /* 1: pairs (2i, 2i+1); 0: pairs (i, i + rot_dim/2) */
  int scaling;       /* MONO_ROPE_* */
  double theta;      /* > 1, e.g. 10000 */
  double factor;     /* context stretch, >= 1 (unused by MONO_ROPE_NONE) */
  double beta_fast, beta_slow; /* YaRN: turns over orig_context at the ramp's ends, e.g. 32 and 1 */
  int orig_context;  /* YaRN: the context length before the stretch */
  double attn_factor; /* multiplies the rotated values; 0 = 1, for YaRN 0.1 ln(factor) + 1 */
} mono_rope_config;

/* A prepared rotation: a plain value, filled by mono_rope_init and passed by
 * pointer; nothing on the device belongs to it.  turns[i] = revolutions a
 * position of pair i, in binary64: the kernels reduce position x turns to one
 * revolution in binary64, so far positions keep full precision. */
typedef struct {
  int rot_dim, offset, interleaved;
  double factor;
  double turns[128];
} mono_rope;

/* Host only.  Refuses with every reason. */
int mono_rope_init(const mono_rope_config* cfg, mono_rope* out);

/* out[t][h] = x[t][h] rotated to position pos[t], for tokens x heads rows of
 * head_dim values: with a = 2 pi turns_i pos, c = factor cos a, s = factor sin a
 *   (y1, y2) = (c x1 - s x2, s x1 + c x2)
 * and the other dimensions copied.  transpose = 1 applies the transposed map
 * (s negated): the gradient of the rotation, and for factor 1 its inverse.
 * pos[t] < 0 marks a padding row: out is left as it was.  Computed in fp32,
 * rounded once.  dtype MONO_F32 | MONO_BF16 for both.  out may be x itself
 * (same strides); any other overlap of their address ranges is refused, and so
 * is an out whose rows overlap.  heads <= 65535, head_dim <= 1024. */
int mono_rope_apply(const mono_rope* rope, int tokens, int heads, int head_dim, int dtype, const void* x,
                    int64_t x_token, int64_t x_head, const int* pos, void* out, int64_t out_token, int64_t out_head,
                    int transpose, void* stream);

/* ---------------------------------------- the paged 8-bit cache, attention */

typedef struct {
  int q_heads;    /* a multiple of kv_heads, q_heads / kv_heads <= 128 */
  int kv_heads;
  int head_dim;   /* 64, 128 or 256 */
  int page_size;  /* tokens a page: 16, 32, 64 or 128 */
  int num_pages;  /* pages of each cache that a call names */
  int max_seqs;   /* sequences a call may pass, <= 4096 */
  int max_pages;  /* columns of the page table */
  int max_new;    /* new tokens a sequence that attend may pass, 1..8 */
  int dtype;      /* MONO_F32 | MONO_BF16: q, k, v and the output */
  float scale;    /* logits = scale q k; 0 = 1 / sqrt(head_dim) */
  int window;     /* a token sees itself and window - 1 tokens before it; 0 = all before it */
  int device;
} mono_attn_config;

/* One layer's cache, caller-owned device memory, any content at first:
 *   k, v             e4m3 codes [num_pages][kv_heads][page_size][head_dim], 16-byte aligned
 *   k_scale, v_scale fp32 [num_pages][kv_heads]: value = code x scale, one
 *                    scale for each page (block of tokens) and head */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
} mono_kv_cache;

/* q, k, v or the output: element (s, j, h, d) at p[s seq + j token + h head + d] */
typedef struct {
  void* p;
  int64_t seq, token, head;
} mono_rows;

/* The sequences of a call, device memory:
 *   lens  int32 [seqs]: tokens of the sequence, the new ones included
 *   n_new int32 [seqs] or NULL: how many of the call's `width` rows are new
 *         tokens (NULL: all).  Row j < n_new is the token at position
 *         lens - n_new + j; rows behind it are padding.  n_new <= 0: a padding
 *         sequence, its other entries are not read.
 *   table int32 [seqs][max_pages]: entry i is the page of tokens
 *         [i page_size, (i + 1) page_size); entries behind the sequence's end
 *         (and, with a window, before its first visible token) may hold anything.
 * A page id outside [0, num_pages), lens above max_pages x page_size or below
 * 0, or n_new above width is recorded for mono_attn_query_error; the tokens
 * concerned are left out (with n_new above width the whole sequence: its pages
 * and its rows stay as they were) and nothing outside the buffers is touched. */
typedef struct {
  int seqs;
  int width;
  const int* lens;
  const int* n_new;
  const int* table;
} mono_seqs;

typedef struct {
  int grid;               /* CTAs of an attend launch */
  int64_t scratch_bytes;  /* plan-owned device memory */
} mono_attn_info;

typedef struct {
  int code;  /* 0 or MONO_ERR_BAD_INDEX */
  int what;  /* 1 a page id, 2 a length, 3 a number of new tokens */
  int seq;   /* the sequence */
  int value; /* what stood there */
} mono_attn_status;

typedef struct mono_attn_plan_s mono_attn_plan_t;

/* Validate cfg, check the device and allocate the plan's scratch (partial
 * results and arrival counters of attend, the error word).  A plan serves any
 * number of layers' caches.  Calls on one plan that overlap in time share its
 * scratch: order them on one stream or with events (graphs captured on one
 * plan may be replayed in any order, one at a time); use a plan for each
 * concurrent stream.  mono_attn_append uses no scratch. */
int mono_attn_plan(const mono_attn_config* cfg, mono_attn_plan_t** out);

/* Write each sequence's new keys (rotated to their positions when rope is not
 * NULL) and values to its pages.  Per touched page and head, over the new
 * tokens' finite values:
 *   s' = max(amax / 448, 2^-126), and not below the page's scale s when the
 *        page holds older tokens of the sequence (position below the first new one);
 *        NaN if that scale is, and then so are the new codes
 *   code = e4m3(x / s'), nearest, ties to even, saturating (infinities too); NaN stays NaN
 *        (the rotated key x in binary64: codes are rounded once)
 *   older codes become e4m3(code s / s') where s' > s
 * Slots behind the new tokens keep their bytes, and the scale of an untouched
 * page stays.  A page that a call writes stands once in the call's tables (a
 * page that is only read, as a shared prefix by attend, may stand in many).
 * width is not limited by max_new.  Tokens at negative positions (lens <
 * n_new) are not written. */
int mono_attn_append(mono_attn_plan_t* plan, const mono_kv_cache* cache, const mono_seqs* seqs, const mono_rows* k,
                     const mono_rows* v, const mono_rope* rope, void* stream);

/* out(s, j, h) = sum_t softmax_t(scale q(s, j, h) k_t) v_t over the cached tokens
 * t that row j sees: t <= its position, and t > position - window.  q comes
 * rotated; the new tokens' keys and values are in the cache already (append
 * comes first).  A row that sees nothing gives 0 (lse -infinity).  Rows j >=
 * n_new of a sequence, and padding sequences, leave out and lse as they were.
 * What lies in unseen tokens (NaN included) has no effect.  The address ranges
 * of q and out may not meet, nor rows of out each other.  lse: fp32
 * [seqs][width][q_heads] contiguous, or NULL: the log of the sum of exp(logits).
 * Sums and softmax statistics are fp32; probabilities enter the products with
 * 11 bits (MONO_F32: 22) down to 2^-29 of the row's largest, below it in steps
 * of 2^-39.  q enters with 11 bits (MONO_F32: 22) of fp16's range below each
 * row's largest; rows whose largest is below 2^-86 keep fewer.  Values may have
 * any magnitude for which the sum of exp(logit - largest) |v| stays below fp32's
 * end; MONO_BF16 takes page scales below 2^-111 in steps of 2^-134. */
int mono_attn_attend(mono_attn_plan_t* plan, const mono_kv_cache* cache, const mono_seqs* seqs, const mono_rows* q,
                     const mono_rows* out, float* lse, void* stream);

/* Synchronise the plan's device, read the first recorded bad index into *st
 * (may be NULL) and clear it.  Returns 0 or MONO_ERR_BAD_INDEX. */
int mono_attn_query_error(mono_attn_plan_t* plan, mono_attn_status* st);

int mono_attn_get_info(const mono_attn_plan_t* plan, mono_attn_info* info);
void mono_attn_destroy(mono_attn_plan_t* plan);

/* ------------------------------------------------------ 4-bit projections */

enum {
  MONO_INT4 = 4  /* unsigned 4-bit codes q, value (q - zero) x scale; beside MONO_MXFP4 of mono_ffn.h */
};

typedef struct {
  int n_out;        /* rows of W, 1..2^30 */
  int n_in;         /* columns of W, a multiple of group */
  int format;       /* MONO_INT4 | MONO_MXFP4 */
  int group;        /* inputs a scale: a multiple of 32; 32 for MONO_MXFP4 */
  int scale_dtype;  /* MONO_INT4: MONO_F32 | MONO_BF16; MONO_MXFP4: ignored (e8m0) */
  int zeros;        /* MONO_INT4: 1 = zero points at packing, 0 = zero is 8 */
  int dtype;        /* MONO_F32 | MONO_BF16: x and y */
  int device;
} mono_proj_config;

typedef struct mono_proj_plan_s mono_proj_plan_t;

typedef struct {
  int cluster;           /* CTAs that share an output block's inputs */
  int64_t packed_bytes;  /* plan-owned packed weights */
} mono_proj_info;

int mono_proj_plan(const mono_proj_config* cfg, mono_proj_plan_t** out);

/* Repack W once into the plan's kernel layout (blocks of 64 outputs x 32
 * inputs in the order that the tensor-core fragments take them):
 *   codes  uint8 [n_out][n_in / 2], two codes a byte, the even input in the low nibble
 *   scales [n_out][n_in / group] in scale_dtype, or e8m0 bytes (255 = NaN)
 *   zeros  uint8 [n_out][n_in / group], 0..15 (low nibble taken), or NULL when cfg.zeros is 0
 * Asynchronous on `stream`; the inputs may be freed after the stream reaches
 * this point, and steps on other streams must wait for it. */
int mono_proj_pack(mono_proj_plan_t* plan, const void* codes, const void* scales, const void* zeros, void* stream);

/* y[r][n] = sum_k x[r][k] W[n][k] for rows 0..8 (0 is a no-op), rows x_row
 * and y_row elements apart.  Products are exact and sums fp32; y is rounded
 * once.  x enters with 11 bits below each row's largest finite magnitude that one
 * warp reads down to 2^-29 of it (bf16 is exact there), MONO_F32 with 22, and
 * below 2^-112 in steps of 2^-150.  An infinity in x gives what the sum of
 * products has: infinities of the weights' signs, NaN where a weight is zero or
 * two of them meet.  y may not overlap x.  Uses no scratch: calls on one plan
 * may overlap. */
int mono_proj_step(mono_proj_plan_t* plan, int rows, const void* x, int64_t x_row, void* y, int64_t y_row,
                   void* stream);

int mono_proj_get_info(const mono_proj_plan_t* plan, mono_proj_info* info);
void mono_proj_destroy(mono_proj_plan_t* plan);

/* Every reason of the last failure of a call of this header on this thread. */
const char* mono_attn_last_error(void);

#ifdef __cplusplus
}
#endif
#endif
