// kv_cache.cuh -- where the paged key/value cache keeps a token (the layout
// is described in include/attn_paged.h).
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

}  // namespace attnpipe
