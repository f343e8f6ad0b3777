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
 *     (documents) and, for prefill, a bidirectional prefix;
 *   - pgdx_fork_rows, pgdx_copy_pages, pgdx_compact_pages: table rows that
 *     share pages -- forked, reordered (beam search), cut back and released
 *     over reference counts -- page copies, and the pool's compaction;
 *   - pgdx_shared_decode: decode attention of rows that share their first
 *     pages, which are read once for all of them.
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

/*
 * fork_rows -- makes each table row a copy of an old row (its parent), cut to the
 * positions it keeps, over reference-counted pages: forks (parents[r] = the
 * row forked), beam search's reordering (any map), releases (parents[r] = -1) and
 * cuts (keep) in one call.
 *   rows         R in 0 .. 8192; max_pages_per_row: W, R * W <= 2^30.
 *   table        int32 [R][W], read and rewritten in place: row i's first
 *                ceil(lengths[i] / 64) entries are its pages.
 *   lengths      int32 [R]: positions of each row in the cache.
 *   parents      int32 [R]: the old row that row r continues, or -1: row r gets none.
 *   keep         int32 [R]: row r keeps its parent's first keep[r] positions (all
 *                of them if it has fewer; below 0: none), or NULL: all.
 *   shares       int32 [num_pages], read and written: how many rows hold each page
 *                beyond the first (0: held once, or free; pgdx_assign_pages hands
 *                out free pages, whose shares are 0).
 *   free_pages   int32 [num_free], free_head: the list as for pgdx_assign_pages, here
 *                read and written: pages are taken from index *free_head on and
 *                given back below it.
 * Row r gets the length n = min(lengths[parent], keep) and the parent's first
 * ceil(n / 64) entries (entries past them stay as they are).  Shares follow.
 * Pages that no row holds any more are given back, first of all, in the order
 * of the old entries (row by row) that held them first: to indices *free_head - their
 * count .. *free_head - 1.  Then a last page in part use (n % 64 != 0) becomes the
 * row's own, for its next positions to be written there: where all that hold the
 * page hold it so, the lowest row keeps it; each other row takes the next free
 * page, in row order, and leaves the copy to pgdx_copy_pages:
 *   sources, targets, counts  int32 [R]: row r's page to copy from and to and its
 *                positions in use (n % 64), or -1, -1, 0.
 *   new_lengths  int32 [R]: n.
 *   free_head_out  int32 [1]: the list's next page afterwards.
 * Outputs must not overlap each other or an input (table, shares and free_pages
 * count as outputs).
 * Device errors (PGD_EDEVICE_BOUNDS): a length outside [0, 64 W] (taken as 0); a parent
 * outside [-1, R) (taken as -1); an entry outside the pool (its page is not
 * counted); a page given back, or left for a copy of it, by more rows than hold it by its
 * shares; no page, or one outside the pool, for a last page's copy, or a last page outside
 * the pool: the row loses that page, its new length is rounded down to whole pages; a
 * *free_head outside [0, num_free]: nothing is taken or given back; a list with too few
 * places below *free_head: the pages without one are lost to it.
 * PGD_ECUDA leaves table, shares and free_pages as they were, the other outputs undefined.
 */
PGD_API int pgdx_fork_rows(int32_t rows, int32_t max_pages_per_row, int32_t num_pages,
                           int32_t* table, const int32_t* lengths, const int32_t* parents,
                           const int32_t* keep, int32_t* shares, int32_t* free_pages,
                           int32_t num_free, const int32_t* free_head, int32_t* new_lengths,
                           int32_t* sources, int32_t* targets, int32_t* counts,
                           int32_t* free_head_out, pgd_stream_t stream);

/*
 * copy_pages -- copies the first counts[i] positions of page sources[i] to page
 * targets[i], for all kv heads, in the K and V pools of each layer.
 *   dims         num_kv_heads, head_dim, num_pages and layout (PAGE_MAJOR or HEAD_MAJOR,
 *                else PGD_EUNSUPPORTED) of every pool; the rest is not used but checked.
 *   layers       L >= 0; k_pools, v_pools: host arrays of L device pointers.
 *   copies       n >= 0; sources, targets, counts: int32 [n]; counts NULL: 64.
 * A negative source or target: no copy.  A page that is a target must not be named
 * by another copy (pgdx_fork_rows' and pgdx_compact_pages' copies never are).
 * Device errors: a page outside the pool or a count outside [0, 64]
 * (PGD_EDEVICE_BOUNDS): that copy is left out.
 */
PGD_API int pgdx_copy_pages(const pgd_dims* dims, int32_t layers, void* const* k_pools,
                            void* const* v_pools, int32_t copies, const int32_t* sources,
                            const int32_t* targets, const int32_t* counts, pgd_stream_t stream);

/*
 * compact_pages -- moves held pages to the lowest free ones: with k counting from
 * 0, the k-th highest page held by a row goes to the k-th lowest page listed as
 * free, as long as that is lower and k < max_moves.  Pages neither held nor listed
 * stay as they are.
 *   table, lengths, shares, free_pages, free_head: as for pgdx_fork_rows; every row that
 *                holds pages is in the table.
 *   new_table    int32 [R][W]: the table with the pages' new names (entries past a row's
 *                pages copied); new_shares int32 [num_pages]; new_free int32
 *                [num_free]: from *free_head on the free pages, lowest first,
 *                before it copied.  Each may be its input.
 *   sources, targets  int32 [max_moves]: the copies, for pgdx_copy_pages; -1 past the last.
 *   end          int32 [1]: 1 + the highest page held afterwards (0: none).
 *   workspace    pgdx_compact_workspace_bytes(num_pages) bytes.
 * Otherwise outputs must not overlap each other or an input.
 * Device errors (PGD_EDEVICE_BOUNDS; nothing is moved then): a length outside [0, 64 W], an
 * entry or a listed page outside the pool, a page listed twice or both listed and
 * held, a *free_head outside [0, num_free].
 */
PGD_API size_t pgdx_compact_workspace_bytes(int32_t num_pages);
PGD_API int pgdx_compact_pages(int32_t rows, int32_t max_pages_per_row, int32_t num_pages,
                               const int32_t* table, const int32_t* lengths,
                               const int32_t* shares, const int32_t* free_pages, int32_t num_free,
                               const int32_t* free_head, int32_t max_moves, int32_t* new_table,
                               int32_t* new_shares, int32_t* new_free, int32_t* sources,
                               int32_t* targets, int32_t* end, void* workspace,
                               size_t workspace_bytes, pgd_stream_t stream);

/*
 * shared_decode -- pgd_paged_decode_attention (k_new and v_new NULL) or
 * pgd_paged_decode_step (both given), full attention, for rows in groups that share
 * their first pages: the rows b of group g, group_starts[g] <= b < group_starts[g + 1],
 * hold the same first group_pages[g] pages, which are read once for all of them (by the
 * table row of any of them; rows that are inactive, of positions < 0, or whose position is
 * in error may hold others).
 *   groups       S in 0 .. 8192; group_starts int32 [S + 1], not decreasing, in [0, rows];
 *                group_pages int32 [S].  Rows in no group are read on their own.
 *   dims         rows at most 65535; layout PAGE_MAJOR or HEAD_MAJOR (else PGD_EUNSUPPORTED).
 *   workspace    pgdx_shared_decode_workspace_bytes(dims, groups) bytes (0 for dims or groups
 *                that the call refuses).
 *   opts         kernel: PREFILL_UMMA (the groups' pages once), TENSOR_CORE (every row by itself,
 *                by its own table entries, without a look at the groups) or AUTO (TENSOR_CORE where
 *                all rows' tables, whatever of their width is in use, come to 128 MB of pages at
 *                most); else PGD_EUNSUPPORTED.  For short rows in wide tables and for rows that
 *                share nothing TENSOR_CORE is the faster one to ask for.  pages_per_split is not
 *                used.
 * Everything else, inactive rows among it, as there.  A step writes its rows' keys and
 * values to pages of their own: two rows must not hold the page of their positions
 * together.  Device errors (PGD_EDEVICE_BOUNDS, the rows concerned give zeros): a row whose
 * position is beyond its table and, with PREFILL_UMMA, starts that decrease or lie outside
 * (all rows), group_pages outside [0, max_pages_per_row] (its rows), a row whose position is
 * in its group's pages: a step leaves these rows unwritten.  A page outside the pool: a step
 * leaves the row unwritten where that is a page of its own (with TENSOR_CORE: of its last
 * split, as pgd_paged_decode_step), and writes it where it is one of the group's (of a
 * split before).
 */
PGD_API size_t pgdx_shared_decode_workspace_bytes(const pgd_dims* dims, int32_t groups);
PGD_API int pgdx_shared_decode(const pgd_dims* dims, int32_t groups, const int32_t* group_starts,
                               const int32_t* group_pages, const void* q, const void* k_new,
                               const void* v_new, void* k_pool, void* v_pool,
                               const int32_t* table, const int32_t* positions, const float* sinks,
                               float scale, void* out, void* workspace, size_t workspace_bytes,
                               const pgd_decode_options* opts, pgd_stream_t stream);

/* As pgd_get_device_error, for this library's error word. */
PGD_API int pgdx_get_device_error(pgd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PGD_EXT_H_ */
