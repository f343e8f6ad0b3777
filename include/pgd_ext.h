/*
 * pgd_ext.h -- C ABI of libpgd_ext: the rest of a serving step around the
 * paged attention of pgd.h, for GB300 (sm_103a).
 *
 *   - pgdx_assign_pages: the step's block-table entries, slots, rows and
 *     positions, made on the GPU from the requests' lengths;
 *   - pgdx_rotary_append: rotary positions (half or interleaved pairs, part of
 *     the head, scaled frequencies) on q and k, fused with the paged append;
 *   - pgdx_paged_decode, pgdx_paged_prefill: the attention of pgd.h with a
 *     tanh score cap, a distance bias, a first visible key per token
 *     (documents) and, for prefill, a bidirectional prefix.
 *
 * The conventions are those of pgd.h: its types, dims, options, status codes,
 * layouts, alignment (16 bytes for bf16 tensors and the workspace; int32 and
 * fp32 arrays need their natural alignment), inactive rows and device errors.
 * Calls are asynchronous on `stream`; arguments are checked on the host, and a
 * non-zero return means nothing was enqueued.  All pointers are device
 * pointers owned by the caller, except `dims`, `opts`, `score`, `config` and
 * `rotary`, which are host structs read before the call returns.  Calls are
 * captured into CUDA graphs as they are; two graphs (or calls) that can run at
 * the same time need workspaces and outputs of their own.  The library's
 * sticky device error word is its own: pgdx_get_device_error.
 */
#ifndef PGD_EXT_H_
#define PGD_EXT_H_

#include "pgd.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * assign_pages -- block-table entries and slot maps from request lengths (the
 * pages' serving loop hands prefill_paged / step_paged its table, rows,
 * positions and slots: Mistral 7B Instruct v0.3 model files,
 * src/attention.linnet; this makes them without a trip to the host).
 *   requests     R >= 0; max_pages_per_row: table width W >= 1; num_pages: the
 *                pool's pages; num_tokens: P >= 0, the packed pass's token count
 *                (a fixed one for graphs: the tokens past the requests' own are
 *                padding).
 *   table        int32 [R][W], read and written: request r's pages for its
 *                cached[r] positions are in its first ceil(cached[r] / 64) entries.
 *   cached       int32 [R]: positions of each request already in the cache.
 *   new_tokens   int32 [R]: positions each request gets in this pass (0: none).
 *   free_pages   int32 [num_free]: pages to hand out, from index *free_head on
 *                (free_head NULL: from 0).
 * In request order, request r takes ceil((cached + new) / 64) - ceil(cached /
 * 64) pages from the list into its next table entries (entries past them stay
 * as they are), and its new tokens take the next new_tokens[r] places of the
 * packed pass:
 *   rows, positions, slots  int32 [P]: table row, position and pool slot (page
 *                * 64 + position % 64) of each token; padding tokens get row 0,
 *                position -1 and slot -1, which the other calls skip.
 *   starts       int32 [R + 1]: first token of each request, then the count of
 *                the tokens (each at most P).
 *   lengths      int32 [R]: cached + new of the requests served, else cached.
 *   free_head_out  int32 [1]: the index after the last page handed out.
 * The outputs, the table among them, must not overlap each other or an input.
 * Device errors (PGD_EDEVICE_BOUNDS, the first wins): a negative length, a
 * request longer than its table row, too few free pages or places in the pass
 * left for a request: it is not served -- no page, no table entry, its places
 * in the pass (if any) padding, its length as it was.  After a request that
 * found too few pages or places, only requests that need none of these are served.  A
 * page outside the pool (listed free, or the request's last one in use): the
 * tokens on it get slot -1.  A *free_head outside [0, num_free]: no page is
 * handed out, *free_head_out = *free_head.
 */
PGD_API int pgdx_assign_pages(int32_t requests, int32_t max_pages_per_row, int32_t num_pages,
                              int32_t num_tokens, int32_t* table, const int32_t* cached,
                              const int32_t* new_tokens, const int32_t* free_pages,
                              int32_t num_free, const int32_t* free_head, int32_t* rows,
                              int32_t* positions, int32_t* slots, int32_t* starts,
                              int32_t* lengths, int32_t* free_head_out, pgd_stream_t stream);

/* Frequency scalings of the rotary embedding for contexts past the trained
 * one.  With f_i = theta^(-2 i / rotary_dim), i < rotary_dim / 2: */
enum {
  PGDX_ROTARY_NONE = 0,
  PGDX_ROTARY_LINEAR = 1, /* f_i / factor */
  PGDX_ROTARY_NTK = 2,    /* theta * factor^(rotary_dim / (rotary_dim - 2)) for theta (finite) */
  PGDX_ROTARY_YARN = 3,   /* f_i (1 - r_i) + f_i / factor r_i, the ramp r_i = clamp((i - a) /
                             (b - a), 0, 1) from pair a, which turns beta_fast times over
                             original_positions, to pair b, which turns beta_slow times
                             (a, b = rotary_dim ln(original_positions / (2 pi beta)) /
                             (2 ln theta), rounded outwards unless exact_bounds); cos and sin
                             times 0.1 ln(factor) + 1 unless attention_factor is given
                             (GPT-OSS 20B model files, src/rope.linnet) */
  PGDX_ROTARY_BANDED = 4  /* pairs that turn more than high_band times over
                             original_positions keep f_i, those that turn less than
                             low_band times take f_i / factor, between them linear in turns */
};

typedef struct {
  int32_t rotary_dim;    /* leading dims of each head that are rotated: a multiple of 16 in
                            16 .. 128, at most head_dim (checked by the call) */
  int32_t interleaved;   /* 0: dim i pairs with i + rotary_dim / 2; 1: dims 2i, 2i + 1 */
  int32_t scaling;       /* PGDX_ROTARY_* */
  int32_t exact_bounds;  /* YARN: 1 leaves a and b unrounded */
  double theta;          /* > 1 */
  double factor;         /* >= 1 (LINEAR, NTK, YARN, BANDED) */
  double original_positions;  /* > 0 (YARN, BANDED) */
  double beta_fast, beta_slow;  /* YARN: beta_fast > beta_slow > 0 */
  double low_band, high_band;   /* BANDED: high_band > low_band > 0 */
  double attention_factor;      /* factor of cos and sin; 0: the scaling's own (1, but YARN) */
} pgdx_rotary_config;

/* What pgdx_rotary_append takes: filled once by pgdx_rotary_init. */
typedef struct {
  int32_t rotary_dim, interleaved;
  float factor;       /* of cos and sin */
  int32_t reserved;
  uint64_t turns[64]; /* pair i: turns per position times 2^64, its whole turns dropped, so
                         that position * turns[i] mod 2^64 is the exact phase */
} pgdx_rotary;

/* Fills *rotary from *config (host only).  PGD_EINVAL for a value out of the
 * ranges above, PGD_EUNSUPPORTED for a rotary_dim that is no multiple of 16 in
 * 16 .. 128. */
PGD_API int pgdx_rotary_init(const pgdx_rotary_config* config, pgdx_rotary* rotary);

/*
 * rotary_append -- rotates q and k at each token's position and writes rotated
 * k and v into the pools: pair (x, y) at angle a = position * f_i becomes
 * (x c - y s, y c + x s), c and s = factor times cos a and sin a in fp32, each
 * result rounded once to bf16; dims past rotary_dim are copied.  Phases are
 * exact to 2^-32 turns (and 2^-52 of a frequency) at any int32 position.
 *   dims         rows = P tokens; num_q_heads 0 is not allowed: pass q NULL to
 *                leave q out (num_q_heads is then not used).
 *   q            bf16 [P] rows of [Hq][D] at q_stride values apart, or NULL.
 *   q_out        bf16 [P][Hq][D] contiguous; may be q itself when q_stride ==
 *                Hq * D (in place), and must not overlap it otherwise, nor k_new
 *                or v_new.
 *   k_new, v_new bf16 [P] rows of [Hkv][D] at k_stride, v_stride values apart
 *                (views of one fused projection: strides of (Hq + 2 Hkv) * D).
 *                Strides are multiples of 8 values and at least a row long.
 *   positions    int32 [P], < 0: the token is left alone.
 *   slots        int32 [P] pool slots (< 0: the token is left alone), or NULL
 *                to take them from the table:
 *   table, table_rows, token_rows  int32 [table_rows][max_pages_per_row] and the
 *                table row of each token (NULL: row p for token p, table_rows
 *                is then not used); the table may be NULL with PGD_ROW_MAJOR.
 * Two tokens must not name the same slot.  Device errors: a slot, row, page
 * index or page out of range: PGD_EDEVICE_BOUNDS, the token is left alone (its
 * q_out row too).
 */
PGD_API int pgdx_rotary_append(const pgd_dims* dims, const pgdx_rotary* rotary, const void* q,
                               int64_t q_stride, void* q_out, const void* k_new,
                               int64_t k_stride, const void* v_new, int64_t v_stride,
                               const int32_t* table, int32_t table_rows,
                               const int32_t* token_rows, const int32_t* positions,
                               const int32_t* slots, void* k_pool, void* v_pool,
                               pgd_stream_t stream);

/* How the attention's scores differ from scale * q . k.  For the query at
 * position n and the key at position j:
 *   x_j = softcap * tanh(scale q . k_j / softcap)   (softcap > 0; else scale q . k_j)
 *         - alibi_slopes[h] * |n - j|               (alibi_slopes not NULL)
 * for the keys j with lo <= j <= hi, where hi = max(n, prefix_len - 1) and
 * lo = max(0, first_key, n - window + 1 with a window).  A softcap above 2^50 |scale|
 * is refused (PGD_EUNSUPPORTED), one so small that scale / softcap overflows or
 * above 2^126 too (PGD_EINVAL); slopes are finite and at most 2^90.  The sinks join the
 * denominator as they are, neither capped nor biased.  A token that sees no
 * key (first_key > hi) gives zeros.
 * K may hold anything at positions that a token does not see.  So may V, except
 * that in prefill the tokens of one run (same table row and first key,
 * consecutive positions and places in the pass) need finite V wherever one of
 * them sees it. */
typedef struct {
  float softcap;              /* > 0, or <= 0 for none */
  const float* alibi_slopes;  /* device fp32 [Hq], or NULL */
  const int32_t* first_key;   /* device int32 [rows]: first visible position of each row or
                                 token (the start of its document), or NULL for 0 */
  const int32_t* prefix_len;  /* prefill: device int32 [table_rows], positions of each row that
                                 its tokens see whatever their own (a bidirectional prefix,
                                 <= 0: none); NULL otherwise, and for decode */
} pgdx_score;

/*
 * paged_decode -- pgd_paged_decode_attention (k_new and v_new NULL) or
 * pgd_paged_decode_step (both given) with the scores of *score.  Arguments,
 * workspace (pgd_paged_decode_workspace_bytes), results and device errors as
 * there; with a step, the new token is appended whether or not its row sees
 * it.  opts->kernel: AUTO or TENSOR_CORE (else PGD_EUNSUPPORTED).  At most 65535
 * rows and kv heads (the grid's limit; else PGD_EUNSUPPORTED).
 * score->prefix_len must be NULL.
 */
PGD_API int pgdx_paged_decode(const pgd_dims* dims, const pgdx_score* score, const void* q,
                              const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                              const int32_t* table, const int32_t* positions, const float* sinks,
                              int32_t window, float scale, void* out, void* workspace,
                              size_t workspace_bytes, const pgd_decode_options* opts,
                              pgd_stream_t stream);

/*
 * paged_prefill -- pgd_paged_prefill_attention (k_new and v_new NULL) or
 * pgd_paged_prefill_step (both given) with the scores of *score.  A prefix of
 * more positions than the table row holds is a device error
 * (PGD_EDEVICE_BOUNDS, the row's tokens give zeros); the prefix's keys must be
 * in the pools (or written by this step).  opts->kernel: AUTO (PREFILL_UMMA
 * when the tokens average at least 8 a table row and there is more to do than
 * some 14 us of the per-token kernel, with key parts for few items; else per
 * token), TENSOR_CORE or PREFILL_UMMA (else PGD_EUNSUPPORTED).  TENSOR_CORE takes
 * at most 65535 tokens and kv heads (else PGD_EUNSUPPORTED); AUTO takes more in blocks.
 * Both take weights as a bf16 head and residual, against a reference near the
 * row's maximum: PREFILL_UMMA multiplies V by weights up to 2^24 before it divides
 * (softcap up to 52 without a bias; else 2^8), so |V| up to 2^83 stays in range over
 * a million keys.
 * A token's result may change in its last bits with the tokens beside it in the pass
 * (its weights by 2^-20 of the softcap, or 2^-16, relative): AUTO's kernel and key parts
 * go by the call's sizes, and the 32 (token, head) rows of a PREFILL_UMMA warp choose
 * the forms of the cap and of the bias together.  Equal calls give equal bits.
 */
PGD_API int pgdx_paged_prefill(const pgd_dims* dims, int32_t table_rows, const pgdx_score* score,
                               const void* q, const void* k_new, const void* v_new, void* k_pool,
                               void* v_pool, const int32_t* table, const int32_t* rows,
                               const int32_t* positions, const float* sinks, int32_t window,
                               float scale, void* out, void* workspace, size_t workspace_bytes,
                               const pgd_decode_options* opts, pgd_stream_t stream);

/* As pgd_get_device_error, for this library's error word. */
PGD_API int pgdx_get_device_error(pgd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PGD_EXT_H_ */
