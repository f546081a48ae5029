/*
 * attn_packed.h -- C ABI of packed sequences on GB300 (sm_103a): rotation of
 * queries and keys by positions with several axes (attn_rope_packed),
 * attention of every sequence over its own keys (attn_fwd_packed) and its
 * gradients (attn_bwd_packed).
 *
 * The tokens of all sequences of a batch lie one after the other:
 * q [T_q, H_q, D], k and v [T_k, H_kv, D], and sequence b's are the queries
 * cu_q[b] .. cu_q[b + 1] - 1 and the keys cu_k[b] .. cu_k[b + 1] - 1.  No
 * sequence is padded, and any may be empty.  Tokens before cu[0] and behind
 * cu[B] belong to no sequence: nothing of them reaches a result, and their
 * rows of the outputs stay as they were.
 *
 * cu_q and cu_k are [B + 1] int32 device arrays that the kernels read when
 * they run, so a captured graph can be replayed while they change.  What they
 * hold cannot be checked on the host: an entry below 0, below the one before or
 * above T is taken as the nearest that is in order (the one before, or T) and
 * recorded in the device's status word (attn_device_status):
 * ATTN_ERR_BAD_INDEX.
 *
 * Errors are those of attn.h: arguments are checked on the host before
 * anything is queued.  All calls return once their kernels are queued on
 * `stream`; nothing is allocated.
 */
#ifndef ATTN_GB300_PACKED_H
#define ATTN_GB300_PACKED_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A bf16 [T, H, D] tensor (strides in elements, positive multiples of 8; the
 * last dimension contiguous), 16-byte aligned: a view of a projection's output
 * [T, heads, D] needs no copy.  A dimension of size 1 is never stepped along:
 * its stride is not looked at.  An output's elements must lie apart from one
 * another. */
typedef struct {
  void *data;
  int64_t stride_t, stride_h;
} attn_thd_t;

/* The sizes of a packed attention, each at least 1.  H_q a multiple of H_kv; H_q / H_kv at most
 * 32, or a multiple of 4 up to 128; D 64 or 128; B and H_kv at most 65535. */
typedef struct {
  int B, T_q, T_k;  /* sequences, tokens of the tensors */
  int H_q, H_kv, D;
  int causal;       /* 0 or 1 */
  float scale;      /* any finite value, as attn_fwd's */
} attn_packed_t;

/*
 * Attention: for a sequence of n queries and m keys, query head h and
 * g = h / (H_q / H_kv),
 *
 *     s_ij   = scale * sum_d q[i,h,d] k[j,g,d]
 *     A_i    = { j < m }                   (not causal)
 *              { j < m, j <= i + m - n }   (causal: the queries are the newest
 *                                           of the sequence's tokens)
 *     o[i,h,:]  = sum_{j in A_i} exp(s_ij) v[j,g,:] / sum_{j in A_i} exp(s_ij)
 *     lse[h,i]  = ln sum_{j in A_i} exp(s_ij)
 *
 * A query that sees no key gets o = 0 and lse = -inf.  Where n = m (whole
 * prompts) the causal mask is attn_fwd's.
 *
 *   q, k, v    read
 *   o          [T_q, H_q, D], written; must not overlap an input
 *   lse        [H_q, T_q] fp32, contiguous, written
 *   cu_q       [B + 1] int32, device
 *   cu_k       [B + 1] int32, device, or NULL for cu_q (then T_k = T_q)
 *   workspace  caller-owned device scratch, 256-byte aligned, of at least
 *              attn_packed_workspace_bytes(...) bytes; need not be cleared; not
 *              shared with calls that may run at the same time
 *
 * A first kernel lists the tiles of all sequences, the longest first; the
 * attention kernel (attn_fwd's, over tiles of 256 rows that hold whole groups of
 * query heads) takes them on a persistent grid of one thread block per SM.  Where
 * there are few of them, the keys of long ones are cut into parts, which the thread
 * block that ends last joins; up to 31 short sequences take one kernel only.  The
 * results are deterministic.
 *
 * Arithmetic as attn_fwd's: fp32 accumulation and softmax statistics, the
 * probabilities rounded to bf16 (2^-8) before the second product, whose
 * rounded values are also what O is divided by.  A row's exponentials are taken
 * against a maximum that may lag by 2^8, so sums stay finite while |v| times the
 * sequence's keys stays below 2^119.  An infinity or a NaN in a
 * sequence may reach any row of that sequence, masked places included, but of
 * no other sequence.
 */
attn_status_t attn_fwd_packed(const attn_packed_t *sizes, const attn_thd_t *q,
                              const attn_thd_t *k, const attn_thd_t *v, const attn_thd_t *o,
                              float *lse, const int *cu_q, const int *cu_k, void *workspace,
                              size_t workspace_bytes, attn_stream_t stream);

/* Workspace bytes attn_fwd_packed needs (0 if the sizes are invalid).  It does
 * not depend on the lengths. */
size_t attn_packed_workspace_bytes(const attn_packed_t *sizes);

/*
 * Gradients of attn_fwd_packed (its sizes, bounds and workspace rules): given its
 * inputs, its o and lse, and the gradient dout of o,
 *
 *     P_ij = exp(s_ij - lse_i),  dS_ij = P_ij (dout_i . v_j - dout_i . o_i)
 *     dv_j = sum P_ij dout_i,  dk_j = scale sum dS_ij q_i  (over the group's heads too)
 *     dq_i = scale sum dS_ij k_j
 *
 *   q, k, v, o, lse, dout   read
 *   dq         [T_q, H_q, D], written; dk, dv [T_k, H_kv, D], written; queries
 *              that see no key and keys that no query sees get zeros; they must not
 *              overlap an input or one another
 *   deterministic  0: dq is added up in fp32 in the workspace by atomic
 *              additions, whose order (and so dq's last bit) may differ from run
 *              to run; 1: by a kernel of its own, reproducible bit for bit
 *
 * dk and dv are reproducible in any case.  Rounded to bf16: P and dS before their
 * products, and the results.
 */
attn_status_t attn_bwd_packed(const attn_packed_t *sizes, const attn_thd_t *q,
                              const attn_thd_t *k, const attn_thd_t *v, const attn_thd_t *o,
                              const float *lse, const attn_thd_t *dout, const attn_thd_t *dq,
                              const attn_thd_t *dk, const attn_thd_t *dv, const int *cu_q,
                              const int *cu_k, void *workspace, size_t workspace_bytes,
                              int deterministic, attn_stream_t stream);

/* Workspace bytes attn_bwd_packed needs (0 if the sizes are invalid). */
size_t attn_packed_bwd_workspace_bytes(const attn_packed_t *sizes, int deterministic);

/*
 * Rotates queries and keys by positions with several axes.  The rot_dim / 2
 * pairs of a head's elements fall into `axes` sections, sections[0] pairs
 * first; pair d of section a takes row x = positions[a, t] and column d of the
 * tables, and (u, w) becomes
 *
 *     (u cos[x,d] - w sin[x,d], w cos[x,d] + u sin[x,d])        inverse = 0
 *     (u cos[x,d] + w sin[x,d], w cos[x,d] - u sin[x,d])        inverse = 1
 *
 * rounded once to bf16 from the exact value (where a product is not 0 but below 2^-117, whose last
 * bits fp32 does not reach, from a value that may be off by 2^-148).  The second is the
 * gradient of the first.  One axis is the usual rotation.
 *
 *   q, q_out   [T, H_q, D], read and written (may be the same tensor); both NULL
 *              with H_q = 0
 *   k, k_out   [T, H_kv, D], likewise
 *   positions  [axes, T] int32, contiguous, device.  A token with a position
 *              outside [0, rope_rows) is skipped, its output rows stay as they
 *              were, and the status word gets ATTN_ERR_BAD_INDEX.
 *   sections   [axes], on the host, each > 0, their sum rot_dim / 2; axes 1 to 4
 *   cos, sin   [rope_rows, rot_dim / 2] fp32, device, 16-byte aligned
 *   rot_dim    a multiple of 16 up to D; the other elements pass unchanged
 *   interleaved  0: element d < rot_dim / 2 pairs with d + rot_dim / 2;
 *              1: element 2 d pairs with 2 d + 1
 */
attn_status_t attn_rope_packed(const attn_thd_t *q, const attn_thd_t *q_out,
                               const attn_thd_t *k, const attn_thd_t *k_out,
                               const int *positions, const int *sections, int axes,
                               const float *cos, const float *sin, int rope_rows, int rot_dim,
                               int interleaved, int inverse, int T, int H_q, int H_kv, int D,
                               attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_PACKED_H */
