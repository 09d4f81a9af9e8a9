/*
 * decode_attn_paged.h -- a KV cache kept in pages, for NVIDIA GB300 (sm_103a): decode
 * attention over it and the append that fills it, with pages of 16-bit or of 8-bit
 * elements. It stands beside decode_attn_splitkv.h (caches packed through
 * cu_seqlens_k, or one slab per sequence) and shares its status codes, its layouts,
 * its conventions and its device error word.
 *
 * The cache. Keys and values live in `num_pages` pages of `page_size` tokens; a
 * sequence's tokens 0 .. L_b - 1 are spread over the pages that its row of the block
 * table names, token p in page block_table[b][p / page_size] at slot p % page_size.
 * Pages may be shared for reading (common prefixes) and lie in any order.
 *
 * One decode step is an append, then an attention:
 *
 *     kv_lens += new tokens                       (the caller's own kernel)
 *     decode_attn_paged_append(q, k, v, ...)      rotates, writes the new keys and values
 *     decode_attn_paged(q_out, ...)               attends to everything up to each token
 *
 * Conventions are those of decode_attn_splitkv.h: device pointers of the current
 * device, asynchronous work on `stream`, host checks first (a call that returns
 * anything but DA_OK has enqueued nothing), nothing allocated and nothing kept.
 */
#ifndef DECODE_ATTN_PAGED_H
#define DECODE_ATTN_PAGED_H

#include "decode_attn_splitkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a page besides DA_F16 and DA_BF16: 8 bits (1 sign, 4 exponent and 3
   mantissa bits, largest value 448, no infinity), times one float32 scale per page and
   KV head. */
#define DA_E4M3 2

/* More bits of the device error word (decode_attn_splitkv_get_error). */
#define DA_DEVERR_PAGE 0x4u     /* a block-table entry outside [0, num_pages): its keys and values read as
                                   zeros, and nothing is written through it */
#define DA_DEVERR_POSITION 0x8u /* an appended token's position has no row in cos_sin: the token is left out */

/* Largest batch, and largest page, accepted by the calls below. */
#define DA_MAX_PAGED_BATCH 1024
#define DA_MAX_PAGE_SIZE 1024

typedef struct {
    void* k;          /* device, 16-byte aligned: [num_pages, page_size, Hkv, D] (DA_LAYOUT_VARLEN)      */
    void* v;          /*   or [num_pages, Hkv, page_size, D] (DA_LAYOUT_BHSD), contiguous                */
    float* k_scale;   /* device, float32 [num_pages, Hkv], 4-byte aligned, finite and not negative: */
    float* v_scale;   /*   DA_E4M3 only (else ignored, may be NULL)                                      */
    int num_pages;    /* >= 1 */
    int page_size;    /* a multiple of 16 in [16, DA_MAX_PAGE_SIZE] */
    int Hkv;          /* KV heads, >= 1 */
    int D;            /* head size: 64 or 128 */
    int kv_dtype;     /* DA_F16, DA_BF16 or DA_E4M3 */
    int layout;       /* DA_LAYOUT_VARLEN or DA_LAYOUT_BHSD: the order of tokens and heads in a page */
} da_paged_cache;

/*
 * Workspace of the calls below: bytes for any batch and any lengths with these heads
 * (the split step cuts the whole batch's keys into a bounded number of equal ranges,
 * so the size does not grow with the batch). 0 if an argument is out of range.
 * Its base is 256-byte aligned; its first 256 bytes are the header of
 * decode_attn_splitkv.h (error word first), then come counters that are zero between
 * calls, then partial results. Calls that may overlap on the GPU (other streams, two
 * graphs replayed at once) need a workspace each; calls in stream order share one.
 */
size_t decode_attn_paged_workspace_size(int T_q, int Hq, int Hkv, int D);

/*
 * Zero a workspace's header and counters: once on fresh memory, and again after a
 * DA_DEVERR_TIMEOUT. Enqueued on `stream`. Errors: DA_ERR_INVALID_ARG (NULL or too
 * small for any call), DA_ERR_ALIGNMENT, DA_ERR_CUDA.
 */
da_status decode_attn_paged_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/*
 * Decode attention over the paged cache. For query token t of T_q (the last T_q tokens
 * of the sequence, at positions L_b - T_q + t), head h and KV head h / (Hq / Hkv):
 *
 *     x_j = scale * k_scale * (q . k_j)              j <= L_b - T_q + t
 *     out = sum_j softmax(x)_j * v_scale * v_j,      lse = ln sum_j exp(x_j)
 *
 * with the scales of key j's page and head (1 in 16-bit pages). A token that sees no key
 * gets out = 0 and lse = -inf. Memory in a page behind a sequence's last token may hold
 * anything. A NaN or an infinity among keys or values reaches the tokens that see it and
 * no others, nor other heads. The results do not depend on timing: the same inputs on the
 * same device give the same bits.
 *
 * Scores, maxima and sums are float32. A key's weight is rounded before it meets the value:
 * in 16-bit pages to within 2^-15 of itself (bf16), 2^-21 or 2^-36 of the largest one of its
 * token and head (fp16); in 8-bit pages it times v_scale to fp16, 2^-11 of itself or 2^-32
 * of the largest one. (An infinite value whose weight is below 2^-34
 * of the largest one may give NaN.)
 *
 * The call's arguments are the fields of a struct (host memory, read during the call).
 * Errors (nothing enqueued): DA_ERR_INVALID_ARG, DA_ERR_UNSUPPORTED (D, or a batch
 * above the limit), DA_ERR_ALIGNMENT, DA_ERR_WORKSPACE_TOO_SMALL; DA_ERR_CUDA.
 */
typedef struct {
    const void* q;               /* device, [B, T_q, Hq, D] elements of `dtype`, 16-byte aligned */
    const da_paged_cache* cache; /* host; 16-bit pages hold elements of `dtype` */
    const int32_t* kv_lens;      /* device, int32 [B]: keys of each sequence, the query tokens' own included. A
                                    length below 0 or above max_pages * page_size counts as 0 and sets
                                    DA_DEVERR_SEQLENS */
    const int32_t* block_table;  /* device, int32 [B][table_stride], the first max_pages entries of a row
                                    readable; only the entries of a sequence's own tokens are read */
    int max_pages;               /* >= 1; max_pages * page_size <= 0x7fffff00, and B times that <= 2^35 */
    int table_stride;            /* >= max_pages */
    int B;                       /* in [1, DA_MAX_PAGED_BATCH] */
    int T_q;                     /* in [1, DA_MAX_QUERY_TOKENS] */
    int Hq;                      /* a multiple of the cache's Hkv; B * T_q * Hq * D <= 0x7fffffff */
    int dtype;                   /* DA_F16 or DA_BF16 */
    float scale;                 /* finite */
    void* out;                   /* device, [B, T_q, Hq, D] elements of `dtype`, 16-byte aligned */
    float* lse;                  /* device, float32 [B, T_q, Hq], or NULL */
    void* workspace;             /* decode_attn_paged_workspace_size(T_q, Hq, Hkv, D) bytes, initialised once */
    size_t workspace_bytes;
} da_paged_attn;

da_status decode_attn_paged(const da_paged_attn* args, void* stream);

/* How decode_attn_paged_append rotates the first rot_dim dims of queries and keys. */
typedef enum {
    DA_ROPE_NONE = 0,        /* not at all (cos_sin may be NULL) */
    DA_ROPE_HALF = 1,        /* dim i with dim i + rot_dim / 2 */
    DA_ROPE_INTERLEAVED = 2  /* dim 2i with dim 2i + 1 */
} da_rope;

/*
 * Append new tokens to the paged cache, and rotate their queries. Sequence b's new
 * tokens are rows cu_new[b] .. cu_new[b+1] - 1 of q, k and v; row i of them sits at
 * position p = kv_lens[b] - (cu_new[b+1] - cu_new[b]) + i (kv_lens counts them already).
 * With (c, s) = (cos_sin[p][j], cos_sin[p][rot_dim / 2 + j]) a pair (x, y) of a query or
 * key turns into (x c - y s, y c + x s), in float32; the other dims and the values pass
 * as they are. The queries go to q_out, the keys and values to their pages, rounded to
 * nearest-even once.
 *
 * 8-bit pages. An element is stored as x / s rounded to e4m3, s the scale of its page
 * and head in the cache. The call sets s: with `need` the least power of two 2^e (e >= -126)
 * for which every finite new element of the page and head is at most 448 * 2^e,
 *     s = need             if the new tokens start at the page's first slot
 *     s = max(s, need)     otherwise; where s grew, the page's earlier elements are rounded
 *                          again to the new scale
 * A power of two costs no precision (e4m3 is a floating format, so only the smallest
 * values of a page notice its scale) and makes growing a page's scale exact for all
 * elements but those. +-Inf is stored as +-448 s, NaN as NaN; neither moves the scale.
 *
 * The pages that one call writes must be distinct (no two sequences append to the same
 * page). Arguments and errors otherwise as decode_attn_paged.
 */
typedef struct {
    const void* q;               /* device, T_new rows of Hq heads of D contiguous elements of `dtype`, */
    const void* k;               /*   16-byte aligned, rows q_stride elements apart (a multiple of 8), or */
    const void* v;               /*   NULL: nothing to rotate; k and v alike, with Hkv heads */
    int64_t q_stride, k_stride, v_stride;
    const float* cos_sin;        /* device, float32 [max_pos][rot_dim], 16-byte aligned: cosines, then sines */
    int max_pos;
    int rot_dim;                 /* a multiple of 16 in [16, D] (ignored without rotation) */
    int rope;                    /* da_rope */
    const int32_t* cu_new;       /* device, int32 [B+1], non-decreasing; rows from cu_new[B] on are left alone. (Where it
                                    decreases, that sequence is left out, and so may be others; a row that two of the
                                    rest claim goes to either or to both.) */
    const int32_t* kv_lens;      /* device, int32 [B], the new tokens counted */
    const int32_t* block_table;  /* as above */
    int max_pages;
    int table_stride;
    int B;
    int T_new;                   /* rows that q, k and v hold, >= 0 (0: nothing is enqueued, nor flagged; 8-bit pages:
                                    T_new * Hkv <= 0x1fffffff); a sequence whose rows lie outside them, or
                                    whose kv_lens is smaller than its new tokens or larger than max_pages *
                                    page_size, is left out and sets DA_DEVERR_SEQLENS */
    int Hq;
    int dtype;
    const da_paged_cache* cache;
    void* q_out;                 /* device, rows like q's, q_out_stride elements apart; may be q itself with the
                                    same stride, else it must not overlap q, k or v */
    int64_t q_out_stride;
    void* workspace;             /* its header alone is used (the error word): initialised, 256-byte aligned */
} da_paged_append;

da_status decode_attn_paged_append(const da_paged_append* args, void* stream);

/*
 * decode_attn_paged of a model with a sliding window: the token at position p sees key j where
 * j <= p and (j > p - window or j < sinks): itself and the window - 1 tokens before it, and the
 * sequence's first `sinks` tokens, which stay visible however long it gets. Only pages that hold a
 * key which some token sees are read (block-table entries of the others are not, and may hold
 * anything). window in [1, 0x7fffffff], sinks in [0, 0x7fffffff]; arguments, results, workspace and
 * errors otherwise as decode_attn_paged.
 */
da_status decode_attn_paged_window(const da_paged_attn* args, int window, int sinks, void* stream);

/*
 * Attention of a chunk of new tokens of each sequence over its pages: a prompt, a part of one, a
 * drafted continuation or a single token, in any mixture. As in decode_attn_paged_append sequence
 * b's tokens are rows cu_new[b] .. cu_new[b+1] - 1 of q, and row i of them sits at position
 * p = kv_lens[b] - (cu_new[b+1] - cu_new[b]) + i (kv_lens counts them already, and their keys and
 * values are in the pages). A row sees key j where
 *
 *     j <= p  and  (window = 0  or  j > p - window  or  j < sinks)
 *
 * and gets out and lse as decode_attn_paged defines them; a row that sees no key (p < 0, an empty
 * sequence) gets out = 0 and lse = -inf. Rows that belong to no sequence are left alone, in out and
 * lse alike. What a page holds behind a sequence's end, or block-table entries of pages that no row
 * sees, may be anything. A NaN or an infinity among keys or values reaches the rows that see it and no
 * others, nor other heads. The results do not depend on timing: the same inputs on the same device
 * give the same bits.
 *
 * Scores, maxima, sums and accumulators are float32. A key's weight is rounded once before it meets
 * the value: in bf16 pages to bf16, in fp16 pages to fp16 and in 8-bit pages (with v_scale) to fp16,
 * both lifted by 2^11 towards the top of that type, so that weights count down to 2^-36 of the
 * largest one of the row. Over 8-bit pages queries enter as fp16 scaled by a power of two per row (an
 * element below 2^-28 of its row's largest loses bits). (An infinite value whose weight is below that,
 * and a value of 8-bit pages whose weight without v_scale is below 2^-126, may count as none or give NaN.)
 */
typedef struct {
    const void* q;               /* device, T_new rows of Hq heads of D contiguous elements of `dtype`, 16-byte aligned, */
    int64_t q_stride;            /*   rows q_stride elements apart (a multiple of 8, >= Hq * D)             */
    const da_paged_cache* cache; /* host; 16-bit pages hold elements of `dtype` */
    const int32_t* cu_new;       /* device, int32 [B+1], non-decreasing; a sequence whose rows are not within 0 .. T_new, or
                                    end before they begin, is left out and sets DA_DEVERR_SEQLENS. (A row that two
                                    sequences claim then goes to either or to both.) */
    const int32_t* kv_lens;      /* device, int32 [B], the new tokens counted. A length below 0 or above max_pages *
                                    page_size counts as 0 and sets DA_DEVERR_SEQLENS */
    const int32_t* block_table;  /* as above; an entry outside [0, num_pages) sets DA_DEVERR_PAGE, its keys and values
                                    read as zeros */
    int max_pages;
    int table_stride;
    int B;                       /* in [1, DA_MAX_PAGED_BATCH] */
    int T_new;                   /* rows that q and out hold, >= 0 (0: nothing is enqueued) */
    int Hq;                      /* a multiple of the cache's Hkv; T_new * Hq / Hkv <= 0x3fffffff */
    int dtype;                   /* DA_F16 or DA_BF16 */
    float scale;                 /* finite */
    int window;                  /* >= 1, or 0: no limit */
    int sinks;                   /* >= 0 (ignored where window is 0) */
    void* out;                   /* device, rows like q's, out_stride elements apart; no overlap with q */
    int64_t out_stride;
    float* lse;                  /* device, float32 [T_new, Hq], or NULL */
    void* workspace;             /* decode_attn_paged_chunk_workspace_size(Hq, Hkv, D) bytes, initialised once by */
    size_t workspace_bytes;      /*   decode_attn_paged_workspace_init; serves the other calls too, if large enough */
} da_paged_chunk;

/* Workspace of decode_attn_paged_chunk, for any batch and any lengths with these heads; 0 if an argument is out of range. */
size_t decode_attn_paged_chunk_workspace_size(int Hq, int Hkv, int D);

da_status decode_attn_paged_chunk(const da_paged_chunk* args, void* stream);

/*
 * Managing the pages. The block table and the lengths say which pages are in use: page p of the first
 * ceil(kv_lens[b] / page_size) entries of row b. Nothing else is kept, so a sequence is freed by
 * setting its length to 0 (or leaving its row out), and
 *
 *     decode_attn_paged_free_pages     lists the pages that no row uses,
 *     decode_attn_paged_fork           makes rows that continue other rows and share their pages,
 *     decode_attn_paged_compact        moves the pages in use to the front of the cache.
 *
 * They read one table and write another one, which must not overlap it, and can be captured and repeated.
 * A length below 0 or above max_pages * page_size counts as 0 and sets DA_DEVERR_SEQLENS; an entry
 * outside [0, num_pages) is used by no one, is copied as it is, and sets DA_DEVERR_PAGE. The results do not
 * depend on timing.
 */
typedef struct {
    const int32_t* kv_lens;      /* device, int32 [B] */
    const int32_t* block_table;  /* device, int32 [B][table_stride]; only the entries in use are read */
    int max_pages;               /* >= 1; max_pages * page_size <= 0x7fffff00 */
    int table_stride;            /* >= max_pages */
    int B;                       /* in [1, 65536]; B * max_pages <= 0x7fffffff */
    int page_size;               /* a multiple of 16 in [16, DA_MAX_PAGE_SIZE]; the cache's own where there is one */
    int num_pages;               /* >= 1, num_pages * page_size <= 0x7fffff00; the cache's own where there is one */
    void* workspace;             /* decode_attn_paged_pages_workspace_size(num_pages) bytes, initialised once by */
    size_t workspace_bytes;      /*   decode_attn_paged_workspace_init; serves the other calls too, if large enough */
} da_paged_rows;

/* Largest B of the calls below. */
#define DA_MAX_PAGED_ROWS 65536

/* Workspace of the calls below; 0 if num_pages is out of range. */
size_t decode_attn_paged_pages_workspace_size(int num_pages);

/*
 * free_pages[0 .. n-1] = the pages that no row uses, ascending; num_free[0] = n. Entries of free_pages
 * (device, int32 [num_pages]) from n on are left alone.
 */
da_status decode_attn_paged_free_pages(const da_paged_rows* rows, int32_t* free_pages, int32_t* num_free, void* stream);

/*
 * Row i of block_table_out (i < n_out) continues row parents[i]: it gets its length and its pages. Where
 * new_pages[i] >= 0 and the length is no multiple of the page size, new_pages[i] takes the place of the last,
 * partly filled page, and that page's tokens (keys, values and 8-bit pages' scales) are copied to it, so that both
 * rows can be appended to; with new_pages[i] < 0 the last page is shared like the others (one row at most may
 * append to it). A parent outside [0, B) sets DA_DEVERR_SEQLENS and gives a row of length 0; a new page outside the
 * cache sets DA_DEVERR_PAGE and is not written. A last entry outside the cache stays as it is like the others: there is
 * nothing that the new page could hold. Entries behind a row's pages are left alone. The new pages must be
 * distinct, and none of them in use.
 *   parents, new_pages   device, int32 [n_out], n_out in [1, 65536]
 *   kv_lens_out          device, int32 [n_out]; block_table_out device, int32 [n_out][table_out_stride],
 *                        table_out_stride >= max_pages; neither overlaps an input
 *   rows                 page_size and num_pages must be the cache's, a page's keys less than 32 GB (else DA_ERR_UNSUPPORTED)
 */
da_status decode_attn_paged_fork(const da_paged_rows* rows, const da_paged_cache* cache, const int32_t* parents,
                                 const int32_t* new_pages, int n_out, int32_t* kv_lens_out, int32_t* block_table_out,
                                 int table_out_stride, void* stream);

/*
 * With n pages in use, the pages in use from n on move to the free ones before n, in ascending order both, and
 * num_used[0] = n; pages n .. num_pages - 1 are free afterwards. block_table_out (device, int32 [B][table_out_stride])
 * gets the rows' entries with the pages' new numbers; entries behind a row's pages are left alone, and a page that
 * several rows share moves once. The lengths stay as they are.
 */
da_status decode_attn_paged_compact(const da_paged_rows* rows, const da_paged_cache* cache, int32_t* block_table_out,
                                    int table_out_stride, int32_t* num_used, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_ATTN_PAGED_H */
