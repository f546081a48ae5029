/*
 * attn_paged.h -- C ABI of the paged key/value cache on GB300 (sm_103a): new
 * tokens go into it (attn_kv_append), attention reads it (attn_fwd_paged),
 * and it is read back as contiguous tensors (attn_kv_read).
 *
 * The cache is a pool of pages shared by all sequences.  A page holds
 * page_size tokens of every KV head; position x of sequence b lies in slot
 * x % page_size of page block_table[b * max_blocks + x / page_size].  Two
 * sequences may name the same page to share a prefix.  The lengths, the
 * starts and the block table are device arrays that the kernels read when
 * they run, so a captured graph can be replayed while they change.
 *
 * ATTN_KV_BF16: k and v are [num_pages, H_kv, page_size, D] bf16.
 *
 * ATTN_KV_INT4: k and v are [num_pages, H_kv, page_size / 16, 9 D] bytes:
 * blocks of 16 tokens, each 8 D bytes of codes followed by 16 x G bf16 scales
 * [token][G], G = D / 32 (4.5 bits an element).  A group of 32 consecutive elements
 * x of one token and head has the scale s = bf16(max|x| / 7) and the codes
 * c = clamp(rint(x / s), -7, 7) + 8 (8 throughout where s is 0; rint rounds
 * ties to even), and stands for s (c - 8).  A group that holds an infinity or
 * a NaN has a NaN scale: all of it reads as NaN.  Codes are nibbles, the low
 * one first:
 *   keys    element 32 j + 8 t + n of token r: nibble n of the 4-byte word at
 *           byte r D / 2 + (t G + j) 4                 (j < G, t < 4, n < 8)
 *   values  element 32 j + 4 g + i of token r: nibble i of the 2-byte word at
 *           byte (((r / 2) 8 + g) 2 + r % 2) 2 G + 2 j (j < G, g < 8, i < 4)
 * In this order a thread's share of a block is 4 G consecutive bytes and the
 * two tokens of a value pair lie side by side, as the tensor-core fragments
 * of attn_fwd_paged want them; no byte holds elements of two tokens.
 *
 * Errors are those of attn.h: arguments are checked on the host before
 * anything is queued.  What lies on the device cannot be checked there: the
 * kernels check every page number, length and position they read.  A page
 * number outside [0, num_pages) is never followed: attn_kv_append skips that
 * token, attn_kv_read leaves its rows as they were, and attn_fwd_paged treats
 * the keys as masked.  A length or start below 0 or beyond what the block table
 * spans, and a count of new or query tokens below 0 or above S or S_q, is cut to
 * that range; tokens at positions before 0, behind the span or (where they are
 * rotated) behind the rotation table are skipped.  All of these are recorded in
 * the device's status word (attn_device_status): ATTN_ERR_BAD_INDEX.  The start
 * of a sequence without new tokens is not looked at.
 *
 * All calls return once their kernels are queued on `stream`; nothing is
 * allocated.
 */
#ifndef ATTN_GB300_PAGED_H
#define ATTN_GB300_PAGED_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ATTN_KV_BF16 = 0, ATTN_KV_INT4 = 1 } attn_kv_format_t;

typedef struct {
  void *k, *v;            /* the pools, device, 16-byte aligned */
  const int *block_table; /* [B, max_blocks] int32, device */
  int format;             /* attn_kv_format_t */
  int num_pages;
  int page_size;          /* a multiple of 16 */
  int max_blocks;         /* pages a sequence may hold; max_blocks * page_size < 2^30 */
  int B, H_kv, D;         /* D 64 or 128 */
} attn_kv_cache_t;

/* A bf16 [B, H, S, D] tensor with any strides (in elements, multiples of 8;
 * the last dimension contiguous), 16-byte aligned: a view of a projection's
 * output [B, S, heads, D] needs no copy.  A dimension of size 1 is never
 * stepped along: its stride is not looked at. */
typedef struct {
  const void *data;
  int64_t stride_b, stride_h, stride_s;
} attn_bhsd_t;

/*
 * Writes S new tokens of each sequence into the cache, rotating queries and
 * keys by their positions on the way.  Token i of sequence b has position
 * start[b] + i; with new_lens only i < new_lens[b] are tokens, the rest is
 * padding that is not looked at (the q_out rows of padding stay as they
 * were).
 *
 *   q, q_out   [B, H_q, S, D] bf16, read, and contiguous, written: the rotated
 *              queries (q_out may be q->data where q is contiguous); both
 *              NULL with H_q = 0 when there are no queries to rotate
 *   k, v       [B, H_kv, S, D] bf16, read
 *   start      [B] int32, device: tokens already in the cache
 *   new_lens   [B] int32, device, or NULL for S everywhere
 *   cos, sin   [rope_rows, rot_dim / 2] fp32, device, 16-byte aligned: the
 *              rotation of position x is row x; NULL with rot_dim = 0 for none
 *   rot_dim    0, or a multiple of 16 up to D: the elements that are rotated
 *              (the first ones; the others pass unchanged)
 *   interleaved  0: element d < rot_dim / 2 pairs with d + rot_dim / 2;
 *              1: element 2 d pairs with 2 d + 1
 *
 * A pair (a, b) at position x becomes (a cos - b sin, b cos + a sin), rounded
 * once to bf16 from the exact value, and a 4-bit cache quantises that rounded
 * key: the result depends on nothing but the inputs' values.  Slots must be distinct: two tokens of one call in the same
 * slot (two sequences appending to a shared page) leave either, or a mixture.
 */
attn_status_t attn_kv_append(const attn_kv_cache_t *cache, const attn_bhsd_t *q, void *q_out,
                             const attn_bhsd_t *k, const attn_bhsd_t *v, const int *start,
                             const int *new_lens, const float *cos, const float *sin,
                             int rope_rows, int rot_dim, int interleaved, int H_q, int S,
                             attn_stream_t stream);

/*
 * Reads positions start[b] .. start[b] + S - 1 (0 .. S - 1 without start) of
 * every sequence into contiguous k_out, v_out [B, H_kv, S, D] bf16, the layout
 * attn_fwd takes; a 4-bit cache's values s (c - 8) are rounded to bf16.  Rows
 * of positions at or beyond lens[b] stay as they were.
 */
attn_status_t attn_kv_read(const attn_kv_cache_t *cache, void *k_out, void *v_out,
                           const int *lens, const int *start, int S, attn_stream_t stream);

/*
 * Attention of S_q query tokens per sequence over its lens[b] cached keys:
 * O and LSE as attn_fwd's, with S_kv = lens[b].  With causal the queries are
 * the sequence's newest tokens, whose keys are already in the cache: query i
 * of the n_b = q_lens[b] (or S_q) sees the keys j <= lens[b] - n_b + i.  Without,
 * every query sees every key (cross attention over an encoder's states of
 * another length, kept in the cache, is this case).  A query that sees no key
 * gets O = 0 and LSE = -inf.
 *
 *   q          [B, H_q, S_q, D] bf16, read; rotated already
 *   o, lse     [B, H_q, S_q, D] bf16 and [B, H_q, S_q] fp32, contiguous, written;
 *              rows of queries i >= q_lens[b] stay as they were
 *   lens       [B] int32, device: keys of each sequence, the newest tokens' included
 *   q_lens     [B] int32, device, or NULL for S_q everywhere
 *   workspace  caller-owned device scratch, 256-byte aligned, of at least
 *              attn_paged_workspace_bytes(...) bytes; need not be cleared; not
 *              shared with calls that may run at the same time
 *
 * Where the block table spans more than 1024 keys, the work (units of 64 or 128 keys of
 * all sequences) is dealt out evenly to a grid that fills the GPU, whatever the
 * lengths; a sequence that ends up on more than one thread block is merged by a
 * second kernel.  Meant for decoding, where S_q is one or a few tokens: each
 * (H_q / H_kv) * S_q <= 64 query rows of a KV head read the cache once, and more
 * rows read it once for every 64.  A whole prompt is faster through attn_fwd (2048
 * tokens of 32 heads over 8 of 128: 36 us, here 377): from the first token on, a call
 * over the new keys; behind a cached prefix two calls, one without mask over the
 * prefix as attn_kv_read returns it and one causal over the new keys (attn_fwd's mask
 * begins at its first key), joined by their LSE.  attn_fwd takes one S_q and S_kv a
 * call, so sequences of different lengths are calls of their own.  The results are
 * deterministic for given lengths and span of the block table.
 *
 * Arithmetic: fp32 accumulation and softmax statistics.  bf16 cache: for the
 * second product a probability is the sum of two bf16 numbers (off by 2^-16 of it)
 * where (H_q / H_kv) * S_q <= 8, and one (2^-8) with more rows; values up to
 * 3.3e38 (a rounding by 2^-8 may lift larger ones out of bf16's range) give a
 * finite O while scores stay below 2^26 (beyond, an fp32 exponent no longer holds the
 * margin that keeps sums in range).  4-bit cache: the codes are exact in the
 * products, the queries are exact down to 2^-17 of their row's largest element
 * (smaller elements are off by 2^-25 of it at most), and the probabilities times the
 * values' scales are rounded to fp16 (an error of 2^-11 of a key's share in O, or of
 * 2^-30 of the largest value that the query sees, or 2^-90, where that is more).
 */
attn_status_t attn_fwd_paged(const attn_kv_cache_t *cache, const attn_bhsd_t *q, void *o,
                             float *lse, const int *lens, const int *q_lens, void *workspace,
                             size_t workspace_bytes, int H_q, int S_q, int causal, float scale,
                             attn_stream_t stream);

/* Workspace bytes attn_fwd_paged needs (0 if the arguments are invalid);
 * max_keys = max_blocks * page_size, what the block table spans.  It does not
 * depend on the lengths, and stops growing at 512 thread blocks' parts (4.2 MB at
 * up to 8 rows and D = 128).  256 means that none is used (max_keys <= 1024):
 * attn_fwd_paged then takes a NULL workspace too. */
size_t attn_paged_workspace_bytes(int B, int H_q, int H_kv, int S_q, int D, int max_keys);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_PAGED_H */
