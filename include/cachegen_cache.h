/*
 * cachegen_cache.h -- serving a context after the codec has decoded it:
 * pages that hold keys and values in 8 bits, attention of new tokens over
 * them, attention of whole prompts, and the bookkeeping of pages that
 * sequences share.  Part of libcachegen.so.
 *
 * The Guide to CacheGen's deployment notes (integrating with PagedAttention:
 * direct paged buffer injection) hand the decoded context to a server's
 * block-table cache; cg_decode_paged writes such pages in fp16.  The calls
 * here are what that server does next.  The pages describe none of them, so
 * their definitions are the library's own and stand at each call.
 *
 * Conventions, beside those of cachegen.h (device pointers by the caller,
 * nothing allocated, no state kept, every call asynchronous on its stream
 * and usable in a captured graph, argument errors returned at once, errors
 * found on the device set in the status word at the start of the workspace,
 * which each call clears first):
 *   - A page holds block_tokens tokens of every KV head of one layer's K or
 *     V: [n_blocks][H][block_tokens][d], as in cg_decode_paged.  In the
 *     8-bit formats an element is a code, and a float scale [n_blocks][H]
 *     belongs to each page and head: value = code * scale.
 *   - Token t of a sequence is row t % block_tokens of page
 *     table[sequence][t / block_tokens].  A table entry out of [0, n_blocks)
 *     where a page is needed sets CG_ERR_INVALID_ARG; nothing is read or
 *     written through it.
 *   - 8 <= d <= 128, d a multiple of 8.  Pools and the first rows of q, k, v
 *     and out are 16-byte aligned, and their strides are multiples of 8
 *     elements (positive ones at cg_prompt_attend and cg_cross_attend).  A sequence of an
 *     attention call has at most 2^30 positions.
 *   - Lengths, offsets and ids are int32 on the device; every byte offset is
 *     computed in 64 bits.  Every call takes H * block_tokens up to 2^30 and
 *     n_blocks up to 2^28; cg_cache_write takes block_tokens * d up to 2^32
 *     and H up to 32767.
 *   - Scales of pages are not negative; that of a page whose rows
 *     cg_cache_write adds to is 0 or at least 2^-100, as it writes them.
 *     In the attention calls a finite value of V times the number of positions
 *     stays under 2^112: sums of weights up to 2^15 are taken in fp32.
 *   - An array without entries (rows, ids of a call for none) may be NULL.
 *   - The attention calls' waits for their own copies and products are
 *     bounded (about two seconds); a wait that runs out reports
 *     CG_ERR_TIMEOUT, with the meaning that it has in cachegen.h.
 *   - Sums, softmax statistics and scales are fp32.
 */
#ifndef CACHEGEN_CACHE_H
#define CACHEGEN_CACHE_H

#include "cachegen.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { CG_CACHE_F16 = 0, CG_CACHE_E4M3 = 1, CG_CACHE_INT8 = 2 }; /* what a page's elements are */
enum { CG_F16 = 0, CG_BF16 = 1 };                                /* types of q, k, v rows and outputs */

typedef struct {
    int32_t L;            /* layers: the page calls take 2*L pools (K, V of each) */
    int32_t H;            /* KV heads                                     */
    int32_t d;            /* head dim                                     */
    int32_t block_tokens; /* tokens of a page                             */
    int32_t n_blocks;     /* pages of a pool                              */
    int32_t format;       /* CG_CACHE_*                                   */
} cg_cache;

/* ---- writing pages ------------------------------------------------------ */
typedef struct {
    int32_t n_seq;         /* sequences                                    */
    int32_t n_rows;        /* rows of k and v                              */
    int32_t max_new;       /* no sequence brings more rows than this       */
    int32_t dtype;         /* CG_F16 or CG_BF16                            */
    int32_t table_stride;  /* entries of a table row                       */
    int32_t reserved;      /* must be 0                                    */
    int64_t stride_token;  /* elements from one row to the next            */
    int64_t stride_head;   /* and from one head to the next                */
} cg_rows;

/* New keys and values into 8-bit pages.  Rows cu_new[b] .. cu_new[b+1]-1 are
 * sequence b's tokens at positions start[b], start[b]+1, ...  Any layout with
 * a token and a head stride will do: a projection's [n_rows][H][d], or one
 * layer of the codec's [L][2][H][S][d] (stride_token d, stride_head S*d).
 * For each page, head and K or V that gets rows, with Q = 448 (e4m3) or 127
 * (int8) and all operations in fp32, correctly rounded:
 *   fresh = max|x| * (1 / Q) over the new rows (0 where that is under 2^-100);
 *   scale = fresh where the page's first new row is its row 0, else the
 *           larger of the page's scale and fresh;
 *   a code c of a row before the first new one becomes
 *           code(c * (old scale / scale)) where the scale grew;
 *   a new value becomes code(x * (1 / scale)), 0 where scale is 0;
 *   code() rounds to the nearest, halves to even, and saturates.
 * Rows behind the last new one keep their bytes (they are the caller's to
 * ignore).  No two sequences may write the same page.
 *   k_dev, v_dev:         rows as above.
 *   cu_new_dev, start_dev: int32 [n_seq + 1] and [n_seq].
 *   table_dev:            int32 [n_seq][table_stride].
 *   k_pool, v_pool, k_scale, v_scale: one layer's pages and scales.
 *   ws_dev:               256 bytes, 256-byte aligned.
 * Device errors: CG_ERR_NONFINITE (an Inf or NaN, stored as 0 and left out
 * of the maximum); CG_ERR_INVALID_ARG (a bad page; offsets that fall, pass
 * n_rows or bring more than max_new rows, positions that are negative or
 * outside the table: that sequence is left out). */
cg_status cg_cache_write(const cg_cache *cache, const cg_rows *rows, const void *k_dev, const void *v_dev,
                         const int32_t *cu_new_dev, const int32_t *start_dev, const int32_t *table_dev,
                         void *k_pool, void *v_pool, float *k_scale, float *v_scale, void *ws_dev,
                         size_t ws_bytes, void *stream);

/* ---- attention of new tokens over 8-bit pages ---------------------------- */
typedef struct {
    int32_t n_seq;        /* sequences                                    */
    int32_t q_tokens;     /* T, new tokens of each (1, or drafted ones)   */
    int32_t Hq;           /* query heads, a multiple of H                 */
    int32_t dtype;        /* of q and out                                 */
    int32_t table_stride; /* entries of a table row                       */
    float scale;          /* on q . k, finite and positive                */
    int64_t q_stride[3];  /* elements between sequences, tokens and heads */
} cg_attend;

/* Workspace bytes of cg_cache_attend (0 on bad input). */
size_t cg_cache_workspace_bytes(const cg_cache *cache, const cg_attend *attend);

/* For sequence b, new token t and query head h (KV head h / (Hq / H)), over
 * the positions j <= len[b] - T + t (the new tokens are the last T of len[b]
 * and are in the pages already):
 *   s_j = scale * (q . k_j);  lse = log sum exp(s_j);
 *   out = sum exp(s_j - lse) v_j,   k_j, v_j = code * scale of their page.
 * A row that sees no position gives out 0 and lse -inf.  Bytes behind
 * position len[b]-1, and pages that hold none of it, do not matter, whatever
 * they hold.  The weight of a position in the second product, its probability
 * times its page's V scale, is off by at most 2^-23 of itself or 2^-36 of the
 * largest probability times the largest V scale, whichever is more, and by
 * 2^-11 of itself at most (one under 2^-122 of that may count as 0).
 * A call on the same inputs gives the same bits every time; the bits of a
 * sequence may depend on the lengths of the others.
 *   out_dev: [n_seq][T][Hq][d], contiguous;  lse_dev: fp32 [n_seq][T][Hq], or NULL;  len_dev: int32 [n_seq].
 * Device errors: CG_ERR_INVALID_ARG (a bad page: its positions are left out;
 * a length that is negative or passes table_stride * block_tokens: taken as
 * 0 or as that). */
cg_status cg_cache_attend(const cg_cache *cache, const cg_attend *attend, const void *q_dev, const void *k_pool,
                          const void *v_pool, const float *k_scale, const float *v_scale, const int32_t *table_dev,
                          const int32_t *len_dev, void *out_dev, float *lse_dev, void *ws_dev, size_t ws_bytes,
                          void *stream);

/* ---- attention of new tokens whose sequences share a prefix ----------------- */
typedef struct {
    int32_t n_groups;            /* groups, empty ones among them            */
    int32_t n_members;           /* entries of member_dev                    */
    const int32_t *cu_group_dev; /* [n_groups + 1]                           */
    const int32_t *member_dev;   /* [n_members]                              */
    const int32_t *shared_dev;   /* [n_groups]                               */
} cg_groups;

/* Workspace bytes of cg_shared_attend (0 on bad input). */
size_t cg_shared_workspace_bytes(const cg_cache *cache, const cg_attend *attend, const cg_groups *groups);

/* cg_cache_attend for sequences of which some share the pages of a prefix, as
 * they do after cg_pages_fork: a shared prefix is read once for all of its
 * readers.  Sequences member[cu_group[g]] .. member[cu_group[g+1]-1] are in
 * group g, and their rows of the table begin with the same shared[g] pages, all
 * of them full (cg_pages_groups finds groups, and its arrays can be passed as
 * they are).  Arguments, formulas and outputs are those of cg_cache_attend, with
 * one difference: of a shared prefix a weight is off by at most 2^-11 of itself
 * or 2^-31 of the largest probability times the largest V scale, whichever is
 * more.
 * Sequences that are in no group, and those of a group whose first new token
 * does not see its whole prefix, read all of their positions by themselves.  A
 * group of one is slower than none.  Sharing pays from about 500,000 positions of
 * KV heads that are not read again, (members - 1) * shared * block_tokens * H over
 * all groups, or a million where two share (16 readers, 8 KV heads: of 1024 tokens
 * 25 us, cg_cache_attend 17; of 4096 32 and 33; of 16384 37 and 93).  Below that,
 * and for the finer weights, call cg_cache_attend.
 * Pages of a shared prefix hold no e4m3 NaN.
 * Without groups or members it is cg_cache_attend (the arrays may be NULL then).
 * Device errors: as for cg_cache_attend, and CG_ERR_INVALID_ARG for offsets
 * that are negative, fall or pass n_members (no group counts), a shared[g] that
 * is negative or more than a row of the table (that group does not), a member
 * that is no sequence, or named before (that entry does not). */
cg_status cg_shared_attend(const cg_cache *cache, const cg_attend *attend, const cg_groups *groups, const void *q_dev,
                           const void *k_pool, const void *v_pool, const float *k_scale, const float *v_scale,
                           const int32_t *table_dev, const int32_t *len_dev, void *out_dev, float *lse_dev, void *ws_dev,
                           size_t ws_bytes, void *stream);

/* ---- attention of whole prompts ------------------------------------------- */
typedef struct {
    int32_t n_seq;
    int32_t Hq, H, d;     /* query heads, KV heads, head dim; Hq / H <= 128 */
    int32_t dtype;        /* of q, k, v and out                           */
    int32_t max_q, max_k; /* no sequence has more queries / keys than these */
    int32_t n_q, n_k;     /* rows of q, rows of k and v                   */
    float scale;          /* on q . k, finite and positive                */
    int64_t q_stride[2], k_stride[2], v_stride[2]; /* elements between rows and between heads */
} cg_prompt;

/* Workspace bytes of cg_prompt_attend (0 on bad input). */
size_t cg_prompt_workspace_bytes(const cg_prompt *prompt);

/* Causal attention of packed prompts.  Sequence b has queries
 * cu_q[b] .. cu_q[b+1]-1 and keys cu_k[b] .. cu_k[b+1]-1; its queries are the
 * last ones of its keys, so query i of nq sees keys j <= i + nk - nq (a
 * prompt behind a loaded context has nk > nq; where nk < nq the first rows
 * see nothing and give out 0, lse -inf).  Formulas as at cg_cache_attend.
 * Rows of other sequences, and keys that a row does not see, do not matter,
 * whatever they hold.  Probabilities are rounded to the type of the rows for
 * the second product.  An infinite value of v that a row sees makes its output
 * infinite (NaN beside one of the other sign) as long as its weight is at least
 * 2^-30 (f16) or 2^-110 (bf16) of the row's largest; under that it may be NaN.
 * A call on the same inputs gives the same bits every time; the bits of a
 * sequence may depend on the lengths of the others.
 *   out_dev: [n_q][Hq][d], contiguous;  lse_dev: fp32 [n_q][Hq], or NULL;
 *   rows of q outside every sequence get no output.
 * Device errors: CG_ERR_INVALID_ARG (offsets that fall, pass n_q or n_k, or
 * a sequence with more rows than max_q or max_k: that sequence is left
 * out). */
cg_status cg_prompt_attend(const cg_prompt *prompt, const void *q_dev, const void *k_dev, const void *v_dev,
                           const int32_t *cu_q_dev, const int32_t *cu_k_dev, void *out_dev, float *lse_dev,
                           void *ws_dev, size_t ws_bytes, void *stream);

/* ---- attention to states of another length --------------------------------- */
/* Every query of sequence b sees keys k_begin[b] .. k_begin[b]+k_len[b]-1 and
 * no others: the states of an encoder, or a loaded context without the rows
 * that go on from it (out and lse of such a part can be joined with another
 * part's).  Sequences may share keys.  prompt as at cg_prompt_attend (n_k: rows
 * that k and v have; max_k: no k_len is more), with its workspace, its formulas
 * and its rounding of the probabilities, or a finer one; a row without keys
 * gives out 0, lse -inf.  Keys that a sequence does not see do not matter,
 * whatever they hold.  Where max_q * Hq / H is at most 16 the call goes to a kernel
 * for few rows, with the finer rounding (64 sequences of one query: 28 us, else
 * 66): a decoder's step should give the max_q that it has.
 *   cu_q_dev:               int32 [n_seq + 1], as at cg_prompt_attend;
 *   k_begin_dev, k_len_dev: int32 [n_seq];
 *   out_dev, lse_dev:       as at cg_prompt_attend.
 * Device errors: CG_ERR_INVALID_ARG (offsets that fall, pass n_q or bring more
 * than max_q queries; a k_begin or k_len that is negative, a k_len over max_k,
 * keys past n_k: that sequence is left out). */
cg_status cg_cross_attend(const cg_prompt *prompt, const void *q_dev, const void *k_dev, const void *v_dev,
                          const int32_t *cu_q_dev, const int32_t *k_begin_dev, const int32_t *k_len_dev, void *out_dev,
                          float *lse_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* ---- pages that sequences share --------------------------------------------
 * refs[p] counts the table rows that hold page p; 0 is a free page.  Of the
 * first ceil(len / block_tokens) entries of a table row, each holds a page;
 * the others are -1.  A page that holds a sequence's last, partly filled
 * rows belongs to that sequence alone, so that it can be written.  A call
 * that takes pages takes the free ones with the lowest ids, in the order of
 * its sequences.  Where a fork or an extension finds a bad argument or too
 * few pages, or a fork or a compaction that has pages to move a null or
 * misaligned pool or scale array, it changes nothing at all. */
typedef struct {
    int32_t n_seqs;       /* rows of the table                            */
    int32_t table_stride; /* entries of a table row                       */
    int32_t *refs_dev;    /* [n_blocks]                                   */
    int32_t *table_dev;   /* [n_seqs][table_stride]                       */
    int32_t *len_dev;     /* [n_seqs], tokens                             */
} cg_pages;

/* Workspace bytes of the page calls for up to n sequences, or copies, in a
 * call; pages may be NULL for cg_pages_copy.  0 on bad input. */
size_t cg_pages_workspace_bytes(const cg_cache *cache, const cg_pages *pages, int32_t n);

/* Gives sequence seq[i] (distinct ids) the pages for new_len[i] >= its length
 * and sets its length.  Device errors: CG_ERR_INVALID_ARG (an id or length
 * out of range, a sequence named twice), CG_ERR_CAPACITY (too few free
 * pages); nothing is changed then. */
cg_status cg_pages_extend(const cg_cache *cache, const cg_pages *pages, int32_t n, const int32_t *seq_dev,
                          const int32_t *new_len_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* Makes the empty sequences child[i] (distinct) copies of parent[i]: whole
 * pages are shared, a partly filled last page is copied, in all 2*L pools
 * and scales, to a page of the child's own.
 *   pools_dev:  device array of 2*L page pools, as for cg_decode_paged;
 *   scales_dev: device array of 2*L scale arrays [n_blocks][H], or NULL
 *               (fp16 pages have none).
 * Device errors: as for cg_pages_extend, and CG_ERR_INVALID_ARG for a child
 * that has tokens or is some entry's parent, or, where a page is copied, a
 * null or misaligned pool or scale array; nothing is changed then. */
cg_status cg_pages_fork(const cg_cache *cache, const cg_pages *pages, void *const *pools_dev,
                        float *const *scales_dev, int32_t n, const int32_t *parent_dev, const int32_t *child_dev,
                        void *ws_dev, size_t ws_bytes, void *stream);

/* Drops the sequences: their pages lose a reference each, their table rows
 * become -1 and their lengths 0.  An empty sequence, or one named twice, is
 * dropped once.  Device errors: CG_ERR_INVALID_ARG (an id out of range, left
 * out; a bad page in a table row), CG_ERR_CORRUPT (a page that had no
 * reference). */
cg_status cg_pages_free(const cg_cache *cache, const cg_pages *pages, int32_t n, const int32_t *seq_dev,
                        void *ws_dev, size_t ws_bytes, void *stream);

/* Page dst[i] becomes a copy of page src[i] in all 2*L pools and scales.  No
 * dst may be another entry's src or dst.  Device errors: CG_ERR_INVALID_ARG
 * (an id out of range, a null or misaligned pool or scale array: left out). */
cg_status cg_pages_copy(const cg_cache *cache, void *const *pools_dev, float *const *scales_dev, int32_t n,
                        const int32_t *src_dev, const int32_t *dst_dev, void *ws_dev, size_t ws_bytes,
                        void *stream);

/* Moves the live pages to the front: with n_live pages in use, the i-th free
 * page below n_live gets the contents of the i-th page in use from n_live on,
 * in all 2*L pools and scales.  The new counts and table go to refs_out_dev
 * and table_out_dev, which may be the arrays of `pages` themselves; the
 * lengths stay.  n_live_dev (int32) gets n_live, so a server can give back
 * the pools' tail.  Device errors: CG_ERR_INVALID_ARG (a table entry >=
 * n_blocks, or of a free page: kept as it is; where pages move, a null or
 * misaligned pool or scale array: nothing is changed then, and no output but
 * the status is written). */
cg_status cg_pages_compact(const cg_cache *cache, const cg_pages *pages, void *const *pools_dev,
                           float *const *scales_dev, int32_t *refs_out_dev, int32_t *table_out_dev,
                           int32_t *n_live_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* The rows of a step.  Sequence s of the table brings the last new[s] tokens of
 * its len[s] (cg_pages_extend has given it their pages); their rows lie one
 * after the other, sequences in the table's order:
 *   cu_new_dev: int32 [n_seqs + 1], offsets of each sequence's rows;
 *   start_dev:  int32 [n_seqs], the position of its first new token, len - new;
 *   seq_dev, pos_dev, slot_dev: of each of n_rows rows the sequence, the
 *     position and the place, page * block_tokens + position % block_tokens
 *     (int32, int32, int64 [n_rows]; -1 for the rows behind the last one).
 *     Any of them may be NULL.
 * cu_new_dev and start_dev are what cg_cache_write takes, cu_new_dev is also
 * the cu_q of cg_prompt_attend and cg_cross_attend; the places are for rows
 * that go elsewhere (pages in fp16).
 *   ws_dev: 256 bytes, 256-byte aligned.
 * Device errors: CG_ERR_INVALID_ARG (a length that is negative or passes the
 * table, a new[s] that is negative or more than the length: that sequence
 * brings nothing and its start is 0; a bad page: the row's place is -1);
 * CG_ERR_CAPACITY (more than n_rows rows: offsets stop at n_rows). */
cg_status cg_pages_slots(const cg_cache *cache, const cg_pages *pages, int32_t n_rows, const int32_t *new_dev,
                         int32_t *cu_new_dev, int32_t *start_dev, int32_t *seq_dev, int32_t *pos_dev, int64_t *slot_dev,
                         void *ws_dev, size_t ws_bytes, void *stream);

/* Which sequences share a prefix.  The sequences of the table that have at least
 * min_pages whole pages, of which the min_pages-th is the same page, make a
 * group where they are two or more (after forks and compactions they share
 * everything before it, too).  Groups are in the order of their lowest
 * sequences, members in ascending order:
 *   cu_group_dev: int32 [n_seqs / 2 + 1], offsets of the groups' members;
 *   member_dev:   int32 [n_seqs], sequences, -1 behind the last member;
 *   shared_dev:   int32 [n_seqs / 2], whole pages that a group's rows begin with
 *                 alike, 0 behind the last group (whose offsets end alike).
 *   ws_dev: cg_pages_workspace_bytes(cache, pages, n_seqs).
 * Device errors: CG_ERR_INVALID_ARG (a length that is negative or passes the
 * table, or a bad page at min_pages - 1: that sequence is in no group; a bad
 * page elsewhere in a group's rows is alike to none). */
cg_status cg_pages_groups(const cg_cache *cache, const cg_pages *pages, int32_t min_pages, int32_t *cu_group_dev,
                          int32_t *member_dev, int32_t *shared_dev, void *ws_dev, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif
