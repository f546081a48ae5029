/*
 * attn_testing.h -- test hooks for the kernel's failure detection.
 *
 * Every wait inside the fused kernel gives up after a time budget; the CTA
 * then stops, lets its own copies and tensor-core work finish, frees its
 * tensor memory, and records ATTN_ERR_TIMEOUT in the device status word
 * (attn_device_status in attn.h).  The pages describe no failure handling;
 * these hooks exist so that path can be tested without faulting the GPU.
 *
 * attn_fwd_timeout_test runs the same computation as attn_fwd (same
 * arguments and buffers) in the diagnostic instantiation of the kernel, with
 * one difference: the first softmax warpgroup of every CTA that reaches KV
 * block `drop_block` does not signal that its probabilities are ready, so
 * the tensor-core issuer's wait for them runs out after `wait_budget_ns`.
 * A CTA whose sequence has fewer blocks completes normally.  Outputs of a
 * timed-out CTA are unspecified.  `wait_budget_ns` must lie in
 * [1 ms, 2 s]; `drop_block` must be >= 0 (else ATTN_ERR_INVALID_ARG).
 * For tests only.
 *
 * attn_fwd_tail_timeout_test does the same for the split tail of attn_fwd (see
 * attn.h: the last round's tiles split across a cluster of two CTAs).  The
 * call runs the split-tail launch with one difference: no CTA of a pair
 * sends its partner the partial result it has staged, so each CTA's bounded
 * wait for the partner's partial runs out after `wait_budget_ns`.  Both
 * CTAs unwind, reach the cluster barrier at exit and return; the status word
 * reads ATTN_ERR_TIMEOUT.  Returns ATTN_ERR_UNSUPPORTED (nothing launched) when
 * attn_fwd would not split the tail for these sizes on this device;
 * `wait_budget_ns` must lie in [1 ms, 2 s].  Outputs are unspecified.
 * For tests only.
 *
 * attn_bwd_timeout_test runs attn_bwd (same arguments and buffers; the
 * path that computes dQ inside the dK/dV kernel) with one difference: in
 * every dK/dV CTA that reaches work item `drop_item` (its query blocks with
 * work, counted from 0 in the order it walks them), the first elementwise
 * warpgroup does not signal that the item's first half block of P^T and
 * dS^T is stored, so the tensor-core issuer's wait for it runs out after
 * `wait_budget_ns`.  Every role of the CTA unwinds (the dQ read-out warps
 * included), the status word reads ATTN_ERR_TIMEOUT and the gradients are
 * unspecified.  `drop_item` must be >= 0 and `wait_budget_ns` in [1 ms,
 * 2 s] (else ATTN_ERR_INVALID_ARG).  For tests only.
 *
 * attn_fwd_paged_timeout_test runs attn_fwd_paged (attn_paged.h; same arguments
 * and buffers) with one difference: the producer warp of every thread block that
 * gets as far as stage `drop_stage` of its keys and values (counted from 0)
 * does not request it, so the consumers' wait for it runs out after
 * `wait_budget_ns`; every warp stops, the producer once its copies under way
 * are in.  Outputs are unspecified.  `drop_stage` must be >= 0 and `wait_budget_ns` in
 * [1 ms, 2 s] (else ATTN_ERR_INVALID_ARG).  For tests only.
 *
 * attn_fwd_packed_timeout_test and attn_bwd_packed_timeout_test run attn_fwd_packed and
 * attn_bwd_packed (attn_packed.h; same arguments and buffers) with one signal
 * withheld: the forward's first softmax warpgroup does not report its probabilities of
 * block `drop_block` of each of its tiles that has one, and the first elementwise
 * warpgroup of the dK/dV kernel (and, where deterministic, of the dQ kernel) not those of half
 * 0 of the `drop_item`-th query tile (key block) that each thread block gets to (both
 * counted from 0), so that the issuer's wait for them runs out after `wait_budget_ns`, and
 * all roles unwind.  Outputs are unspecified.  Limits of
 * `wait_budget_ns` as above; the other number must be >= 0 (else ATTN_ERR_INVALID_ARG).
 * For tests only.
 *
 * attn_fwd_packed_o_boxes returns how many TMA boxes of 32 rows attn_fwd_packed of these sizes
 * may write a tile's O as, from its first row on (rows are token * R + head, R = H_q / H_kv; the
 * box that begins with a row has min(R, 32) heads of 32 / min(R, 32) tokens), 0 where it
 * writes row by row, or -1 for invalid sizes.  Reads nothing but the sizes.
 *
 * attn_fwd_tail_pairs returns how many tiles attn_fwd splits across CTA
 * pairs for these sizes on the current device (0 when the tail is not
 * split), or -1 for invalid sizes or a device that cannot be queried.
 */

#ifndef ATTN_GB300_TESTING_H
#define ATTN_GB300_TESTING_H

#include "attn.h"
#include "attn_packed.h"
#include "attn_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

attn_status_t attn_fwd_timeout_test(const void *q, const void *k, const void *v, void *o,
                                    float *lse, int B, int H_q, int H_kv, int S_q, int S_kv,
                                    int D, int causal, float scale, int drop_block,
                                    unsigned long long wait_budget_ns, attn_stream_t stream);

attn_status_t attn_fwd_tail_timeout_test(const void *q, const void *k, const void *v, void *o,
                                         float *lse, int B, int H_q, int H_kv, int S_q, int S_kv,
                                         int D, int causal, float scale,
                                         unsigned long long wait_budget_ns, attn_stream_t stream);

attn_status_t attn_bwd_timeout_test(const void *q, const void *k, const void *v, const void *o,
                                    const float *lse, const void *dout, void *dq, void *dk,
                                    void *dv, void *workspace, size_t workspace_bytes, int B,
                                    int H_q, int H_kv, int S_q, int S_kv, int D, int causal,
                                    float scale, int drop_item, unsigned long long wait_budget_ns,
                                    attn_stream_t stream);

attn_status_t attn_fwd_paged_timeout_test(const attn_kv_cache_t *cache, const attn_bhsd_t *q,
                                          void *o, float *lse, const int *lens,
                                          const int *q_lens, void *workspace,
                                          size_t workspace_bytes, int H_q, int S_q, int causal,
                                          float scale, int drop_stage,
                                          unsigned long long wait_budget_ns,
                                          attn_stream_t stream);

attn_status_t attn_fwd_packed_timeout_test(const attn_packed_t *sizes, const attn_thd_t *q,
                                           const attn_thd_t *k, const attn_thd_t *v,
                                           const attn_thd_t *o, float *lse, const int *cu_q,
                                           const int *cu_k, void *workspace,
                                           size_t workspace_bytes, int drop_block,
                                           unsigned long long wait_budget_ns,
                                           attn_stream_t stream);

attn_status_t attn_bwd_packed_timeout_test(
    const attn_packed_t *sizes, const attn_thd_t *q, const attn_thd_t *k, const attn_thd_t *v,
    const attn_thd_t *o, const float *lse, const attn_thd_t *dout, const attn_thd_t *dq,
    const attn_thd_t *dk, const attn_thd_t *dv, const int *cu_q, const int *cu_k, void *workspace,
    size_t workspace_bytes, int deterministic, int drop_item, unsigned long long wait_budget_ns,
    attn_stream_t stream);

int attn_fwd_packed_o_boxes(const attn_packed_t *sizes);

int attn_fwd_tail_pairs(int B, int H_q, int H_kv, int S_q, int S_kv, int D, int causal);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_TESTING_H */
