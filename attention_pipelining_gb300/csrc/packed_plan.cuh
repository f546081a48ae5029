// packed_plan.cuh -- what the plan of packed sequences' work (packed_sm103.cu) shares with the
// attention kernel, which finds its own tile where there are few.
#pragma once

#include "attn_internal.h"

namespace attnpipe {

// Scans of two values at once over the warp's lanes up to this one.
template <typename Op>
__device__ __forceinline__ int2 scan_warp(int2 v, Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const int a = __shfl_up_sync(0xffffffffu, v.x, off), b = __shfl_up_sync(0xffffffffu, v.y, off);
    if (lane >= off) v.x = op(v.x, a), v.y = op(v.y, b);
  }
  return v;
}

// Up to 31 sequences: lane i gets the first query and key of sequence i (the last lanes, the
// ends), in order and within the tensors; true where the arrays were not.  Whole warp.
__device__ __forceinline__ bool warp_bounds(const int* cu_q, const int* cu_k, int B, int T_q,
                                            int T_k, int2& first) {
  const int lane = threadIdx.x & 31;
  const bool same = cu_k == cu_q;
  const int a = lane <= B ? cu_q[lane] : 0, b = lane <= B && !same ? cu_k[lane] : 0;
  first = scan_warp(make_int2(max(min(a, T_q), 0), max(min(b, T_k), 0)),
                    [](int x, int y) { return max(x, y); });
  const bool bad = lane <= B && (a != first.x || (!same && b != first.y));
  if (same) first.y = first.x;
  return bad;
}

// The tile (whole, not a part) at query position `pos` of sequence b, which has `queries`
// queries from q0 on and `keys` keys from k0 on.
__device__ __forceinline__ PackedTile packed_tile_at(int b, int q0, int queries, int k0, int keys,
                                                     int pos, int positions, int causal) {
  PackedTile x;
  x.tok0 = q0 + pos;
  x.rows = min(queries - pos, 2 * positions);
  x.k0 = k0;
  x.k_len = keys;
  x.diag = keys - queries + pos + 1;
  x.n_keys = causal ? min(max(x.diag + x.rows - 1, 0), keys) : keys;
  x.vec0 = packed_vec0(q0, b) + pos;
  x.jb = 0;
  x.n_blocks = (x.n_keys + 127) >> 7;
  x.parts = 1;
  x.part = 0;
  x.slot = 0;
  return x;
}

}  // namespace attnpipe
