// kv_cache.cuh -- where the paged key/value cache keeps a token (the layout
// is described in include/attn_paged.h), and how its kernels are launched.
#pragma once

#include <cstdint>

#include "attn_internal.h"

namespace attnpipe {

// Bytes of 16 tokens of one head's keys (or values): the unit both formats
// are laid out in, contiguous for bf16 as well.
template <int D, bool kInt4>
constexpr int kKvBlockBytes = kInt4 ? 9 * D : 32 * D;

// Byte offset of 16-token block `blk` of page `page`, head h.
template <int D, bool kInt4>
__device__ __forceinline__ long long kv_block_offset(const KvCache& c, int page, int h, int blk) {
  return (((long long)page * c.H_kv + h) * c.blocks_per_page + blk) * kKvBlockBytes<D, kInt4>;
}

// Programmatic dependent launch: the paged kernels are launched so that their
// thread blocks may be made ready before all of the kernel before them in the
// stream has ended (launch_ahead), and touch no global memory before
// wait_for_earlier, after which everything earlier in the stream is complete
// and visible.  Back to back this hides 1 to 2 us of calls that take 5 to 20.
//
// The attention kernel lets the next one (which merges its parts) come as soon as
// its own blocks are all there (allow_later), and so does the append kernel for
// prompts, but not the others.  Large blocks that come onto SMs while
// small ones are still there are placed unevenly, and one that finds no place then
// starts when others end: where the merge kernel let the next call's blocks
// come early, 16 x 16 heads x 2048 keys took 25 us instead of 21, and where the append
// kernel did for single tokens, append and attention of 4 x 8 x 900 keys 13.4 us
// instead of 12.3.
__device__ __forceinline__ void allow_later() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_earlier() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename Params>
cudaError_t launch_ahead(void (*kernel)(Params), dim3 grid, int threads, int smem_bytes,
                         cudaStream_t stream, const Params& params) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem_bytes;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, params);
}

}  // namespace attnpipe
