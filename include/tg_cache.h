/*
 * tg_cache.h -- C ABI of the paged key/value cache operators (sm_100a): block
 * tables and slot maps built on the GPU, keys and values written into pages,
 * ancestor masks of drafted token trees, and the attention of those trees (or
 * of single tokens) over the cache.
 *
 * Together they make one step of decoding, with every length on the device
 * and nothing read back by the host, so that a step can be captured into a
 * CUDA graph:
 *   tg_tree_mask       parents of the drafted tokens -> ancestor masks
 *   tg_tree_attention  drafted tokens attend to the cache and to their ancestors
 *   tg_cache_plan      accepted tokens (or a prompt's) get pages and slots
 *   tg_cache_write     their keys and values go into the pages
 * Drafted keys and values stay in the caller's dense tensors until they are
 * accepted, so rejected tokens never enter the cache.
 *
 * Terms.  A page holds page_size tokens (a power of two, 8 .. 256) of one
 * layer's keys and values.  Request b has lens[b] tokens in the cache; token p
 * lies in page block_tables[b][p / page_size] at row p % page_size; its slot is
 * page * page_size + row.  Drafted (or new) tokens of all requests are packed
 * one request after the other: request b's are rows starts[b] .. starts[b+1] - 1.
 * Free pages stand in a ring of num_pages entries: ring[0] is the index of the
 * first free page's entry in free_pages, ring[1] how many there are.
 *
 * Conventions are those of tg_gemm.h: device pointers on the current device,
 * owned by the caller; asynchronous calls on `stream`; arguments checked on
 * the host before anything is launched (TG_ERR_INVALID_ARG,
 * TG_ERR_MISALIGNED); an output may not overlap an input.  The library
 * allocates nothing here and keeps no pointer; the first call on a device sets it up (its
 * number of SMs, addresses), which may happen inside a stream capture.  Values
 * that only the device knows (lengths, pages, slots, parents) are checked there:
 * what lies out of range is skipped as each entry says, and never read or
 * written through.
 * int32 and int64 arrays are aligned to their element, fp16 / bf16 tensors to
 * 16 bytes, with strides in elements, multiples of 8, and the head dimension
 * contiguous.
 */
#ifndef TG_CACHE_H
#define TG_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "tg_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 16-bit element types of the cache operators. */
enum {
    TG_TYPE_FP16 = 0,
    TG_TYPE_BF16 = 1
};

/* Limits of the cache operators. */
#define TG_CACHE_MAX_BATCH 8192     /* requests of a tg_cache_plan call */
#define TG_TREE_MAX_WORDS 64        /* mask words per token: 2048 tokens a tree */

/* Bits of the status word that tg_cache_plan writes. */
enum {
    TG_PLAN_NO_PAGES = 1,       /* the ring holds fewer pages than are needed       */
    TG_PLAN_TABLE_FULL = 2,     /* a request needs more than max_pages table entries */
    TG_PLAN_BAD_LENGTH = 4,     /* a length is negative or past 2^31 - 1             */
    TG_PLAN_BAD_TOKENS = 8,     /* more tokens than `tokens`, starts not ascending, or a
                                   request appends more than its tokens in the packing */
    TG_PLAN_BAD_RING = 16       /* head or count out of range, or more pages given
                                   back than the ring has room for                   */
};

/*
 * tg_cache_plan -- change the lengths of `batch` requests: pages are taken from
 * the ring or given back to it, block tables extended, and every new token gets
 * its slot and position.
 *
 *   lens          int32 [batch]  tokens in the cache before
 *   add           int32 [batch]  tokens to append (> 0), to drop from the end (< 0; -lens[b]
 *                                releases the request), or 0
 *   starts        int32 [batch + 1] or NULL.  The packing of the new tokens; NULL: request b
 *                                has max(add[b], 0) of them, packed in order
 *   offsets       int32 [tokens] or NULL (needs starts).  Token t of request b becomes number
 *                                offsets[t] of its appended tokens; outside 0 .. add[b] - 1 it
 *                                is not kept.  NULL: its rank in the packing.  Offsets of a
 *                                request's kept tokens are 0 .. add[b] - 1, each once: this is
 *                                the caller's to see to (two tokens with one offset get one
 *                                slot, and a slot whose offset is missing is counted in
 *                                lens_out and written by nobody).
 *   tokens        number of rows of slots and positions
 *   block_tables  int32 [batch][max_pages], rows table_stride apart; new entries are written,
 *                                all others (also those of dropped pages) left as they are
 *   free_pages    int32 [num_pages]  the ring; given-back pages are written behind its tail
 *   ring          int32 [2]      head and count before
 *   lens_out      int32 [batch]  lens + add
 *   ring_out      int32 [2]      head and count after
 *   starts_out    int32 [batch + 1] the packing used (saturated at 2^31 - 1); may be NULL
 *   slots         int64 [tokens] slot of each token, -1: not kept, or behind the last request
 *   positions     int32 [tokens] its position in the request, -1 likewise
 *   status        int32 [1]      0, or TG_PLAN_* bits; then nothing is taken: lens_out = lens,
 *                                ring_out = ring, slots and positions are -1, tables and ring
 *                                entries stay
 *
 * Pages are taken from the head in the order of the requests, and given back in that order
 * behind the tail; pages given back by a call can be taken by the next one.  ring_out and
 * lens_out become ring and lens of the next call.  A page belongs to one request: pages that
 * requests share are the caller's to count, and must not be given back twice.
 * batch <= TG_CACHE_MAX_BATCH, num_pages >= 1, tokens < 2^31.  One kernel.
 */
tg_status_t tg_cache_plan(const int32_t *lens, const int32_t *add, int64_t batch,
                          const int32_t *starts, const int32_t *offsets, int64_t tokens,
                          int32_t *block_tables, int64_t table_stride, int64_t max_pages,
                          int64_t page_size, int32_t *free_pages, int64_t num_pages,
                          const int32_t *ring, int32_t *lens_out, int32_t *ring_out,
                          int32_t *starts_out, int64_t *slots, int32_t *positions,
                          int32_t *status, void *stream);

/*
 * tg_cache_write -- k_cache[slots[t]] = k[t] and v_cache[slots[t]] = v[t] for t < tokens.
 *
 *   k, v      16-bit [tokens][heads][head_dim], row strides token_stride and head_stride
 *             (both tensors the same; tg_cache_write_ex takes v's apart from k's)
 *   slots     int64 [tokens]; a token whose slot is outside 0 .. num_pages * page_size - 1 is
 *             skipped.  Slots that are kept are distinct; if two tokens have the same slot,
 *             each 16 bytes of the row come from one of them.
 *   k_cache, v_cache  16-bit [num_pages][page_size][heads][head_dim] with strides page_stride,
 *             slot_stride and cache_head_stride (both caches the same); written.  They may
 *             be interleaved, but no element belongs to both
 *   head_dim  64 or 128
 *
 * Bits are copied, so any 16-bit type will do.  One kernel.
 */
tg_status_t tg_cache_write(const void *k, const void *v, int64_t tokens, int64_t heads,
                           int64_t head_dim, int64_t token_stride, int64_t head_stride,
                           const int64_t *slots, void *k_cache, void *v_cache, int64_t num_pages,
                           int64_t page_size, int64_t page_stride, int64_t slot_stride,
                           int64_t cache_head_stride, void *stream);

/* tg_cache_write with strides of their own for k and v (keys that a rotation made, values that
   are still a slice of the projection). */
tg_status_t tg_cache_write_ex(const void *k, int64_t k_token_stride, int64_t k_head_stride,
                              const void *v, int64_t v_token_stride, int64_t v_head_stride,
                              int64_t tokens, int64_t heads, int64_t head_dim,
                              const int64_t *slots, void *k_cache, void *v_cache,
                              int64_t num_pages, int64_t page_size, int64_t page_stride,
                              int64_t slot_stride, int64_t cache_head_stride, void *stream);

/*
 * tg_tree_mask -- ancestor masks and depths of drafted token trees.
 *
 *   parents   int32 [tokens]  index of a token's parent among its request's tokens, below its
 *                             own; -1: it follows the context directly
 *   starts    int32 [batch + 1]  packing of the tokens
 *   words     mask words per token, 1 .. TG_TREE_MAX_WORDS
 *   mask      int32 [tokens][words], written: bit j % 32 of word j / 32 is set when token j of
 *             the request is the token itself or one of its ancestors
 *   depth     int32 [tokens], written: number of its ancestors; its position is
 *             lens[b] + depth
 *
 * A token whose parent is not below it or under -1, one past 32 * words, every descendant of
 * such a token, and rows outside every request get an empty mask and depth -1.  One kernel.
 */
tg_status_t tg_tree_mask(const int32_t *parents, int64_t tokens, const int32_t *starts,
                         int64_t batch, int64_t words, int32_t *mask, int32_t *depth,
                         void *stream);

/*
 * tg_tree_attention -- attention of drafted tokens over the cache and over one another:
 *
 *   out[t,h,:] = sum_j softmax_j( scale * q[t,h,:] . key_j ) value_j
 *
 * for every token t of request b, over the lens[b] cached tokens of the request and over its
 * own drafted tokens that the mask shows, with the keys and values of head h / group
 * (group = kv_heads query heads share one).  Scores, maxima and sums are fp32; the probabilities
 * enter the second product in the tensors' type (in fp16, those below 2^-32 of the row's
 * largest are lost); out is rounded once.  A token that sees nothing, or nothing with a score
 * above -inf, gets zeros.  What a token does not see has no influence, not even infinities or
 * NaN there (rejected rows, pages' unused rows).  An infinite value that it sees makes the
 * element infinite, or NaN where the key's weight is 0 (a score of -inf); a cached one (not a
 * drafted one) may also give NaN where its weight is too small for the tensors' type.  Rows of
 * out outside every request are left as they are.
 */
typedef struct {
    int type;                  /* TG_TYPE_FP16 or TG_TYPE_BF16, of all tensors */
    int64_t tokens;            /* rows of q, k, v, out and mask */
    int64_t batch;             /* requests */
    int64_t kv_heads;          /* heads of k, v and the caches */
    int64_t group;             /* query heads per key head, 1 .. 128 */
    int64_t head_dim;          /* 64 or 128 */
    float scale;               /* factor on the scores, 1e-30 .. 1e30; 0: 1/sqrt(head_dim) */
    const void *q;             /* [tokens][kv_heads * group][head_dim] */
    int64_t q_token_stride, q_head_stride;
    const void *k, *v;         /* drafted, [tokens][kv_heads][head_dim] */
    int64_t kv_token_stride, kv_head_stride;     /* of k, and of v unless own_v_strides */
    const void *k_cache, *v_cache;   /* [num_pages][page_size][kv_heads][head_dim] */
    int64_t num_pages, page_size;    /* page_size a power of two, 8 .. 256 */
    int64_t page_stride, slot_stride, cache_head_stride;
    const int32_t *block_tables;     /* [batch][max_pages], rows table_stride apart; an entry
                                        outside 0 .. num_pages - 1 reads as zeros */
    int64_t table_stride, max_pages;
    const int32_t *lens;       /* [batch] cached tokens, clamped to 0 .. max_pages * page_size */
    const int32_t *starts;     /* [batch + 1] packing, clamped to 0 .. tokens */
    const int32_t *mask;       /* [tokens][words], rows mask_stride apart, as tg_tree_mask writes
                                  them; drafted tokens past 32 * words are not seen.  NULL: a
                                  token sees those of its request up to itself (a prompt; key
                                  tiles above the diagonal are computed and masked, so long
                                  prompts take about twice the products of the definition) */
    int64_t words, mask_stride;
    void *out;                 /* [tokens][kv_heads * group][head_dim], written */
    int64_t out_token_stride, out_head_stride;
    void *workspace;           /* tg_tree_attention_workspace_size bytes, 256-byte aligned; any
                                  contents.  Calls that may overlap in time need one each */
    size_t workspace_bytes;
    uint64_t wait_limit_ns;    /* limit of every device-side wait; 0: 2 s.  An expiry is reported
                                  by tg_gemm_check_error as TG_ERR_TIMEOUT */
    int inject;                /* 0, or TG_INJECT_SKIP_FIRST_LOAD: the first CTA skips its first
                                  key load, so that a bounded wait expires (tests) */
    int own_v_strides;         /* nonzero: v has the two strides that follow, not k's */
    int64_t v_token_stride, v_head_stride;
} tg_tree_attention_t;

/* Bytes of workspace for a head width (64 or 128; else 0).  Host only. */
size_t tg_tree_attention_workspace_size(int64_t head_dim);

/*
 * The work of a call is the sum over requests, key heads and pairs of 128-row query tiles
 * of their 128-key tiles; it is divided evenly over the SMs, wherever requests begin and end,
 * and a second kernel joins what was divided (in a fixed order: results do not vary from run
 * to run).  Two kernels; both may be captured into a CUDA graph.
 */
tg_status_t tg_tree_attention(const tg_tree_attention_t *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TG_CACHE_H */
