// attn_tiles.cuh -- tile-level steps shared by the fused kernel and the
// self-test kernels: TMA loads of one 128-row bf16 tile and the two
// tensor-core GEMMs of the attention forward ("PipeThreader: Software-
// Defined Pipelining for Efficient DNN Execution", section A2, Fig. 7:
// load_k / load_v, mma_qk, mma_pv).
//
// Shared-memory tile layout: a [128 rows x D] bf16 tile is stored as D/64
// slabs of [128 rows x 64 columns]; each slab is 128 rows of 128 bytes in
// the 128-byte swizzle (16-byte chunk c of row r sits at chunk c ^ (r % 8)),
// exactly what one TMA load with 128-byte swizzle and a {64, 128} box writes.
// Slabs are 16 KB apart and 1024-byte aligned.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace attnpipe {

constexpr int kTileRows = 128;
constexpr int kSlabBytes = kTileRows * 128;  // one [128 x 64] bf16 slab

template <int D>
struct TileShape {
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr int kSlabs = D / 64;
  static constexpr int kBytes = kTileRows * D * 2;
};

// Loads rows [row0, row0 + 128) of slice z of a [*, rows, D] tensor map into
// `dst` (a tile as above); completion is counted on `bar`.  Rows outside the
// tensor are filled with zeros (and still counted).
template <int D>
__device__ __forceinline__ void tma_load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                              int row0, int z, uint64_t hint) {
#pragma unroll
  for (int s = 0; s < TileShape<D>::kSlabs; ++s)
    tma_load_3d(dst + s * kSlabBytes, map, bar, s * 64, row0, z, hint);
}

// Clears rows [from, 128) of a tile in shared memory that a copy has filled, for
// the tensor core's next read of it (through the async proxy).  Whole warp.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from) {
  const uint32_t base = smem_u32(tile);
#pragma unroll 1
  for (int s = 0; s < TileShape<D>::kSlabs; ++s)
    for (int at = from * 128 + (int)(threadIdx.x & 31) * 16; at < kSlabBytes; at += 512)
      st_shared_v4(base + (uint32_t)(s * kSlabBytes + at), 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// Parts of one piece of work, done by different thread blocks, each of which has written its
// share to global memory: true in the block that came last, for which all of them are
// visible (by loads that do not go through L1).  Whole block; `flag` is in shared memory.
// (The fence before the count orders what the block's threads wrote before the barrier.)
__device__ __forceinline__ bool last_of_parts(int* counter, int parts, volatile int* flag) {
  __syncthreads();   // (the writes are done, and the flag's last use)
  if (threadIdx.x == 0) {
    __threadfence();
    *flag = atomicAdd(counter, 1) == parts - 1;
    __threadfence();
  }
  __syncthreads();
  return *flag != 0;
}

// A part's result of `rows` rows of D floats, as the threads of a warp (a row each) write
// it and the joining threads read it in whole lines: float4 c of row r is float4 c * rows + r.
//
// The joining threads' order, eight floats (c: of float4s 2 c, 2 c + 1) a thread: a warp
// takes eight rows and four pairs of float4s, so that it reads and writes 64 bytes in a
// row at least.  Item i of (rows rounded up to 8) * D / 8.
template <int D>
__device__ __forceinline__ void join_item(int i, int& row, int& c) {
  constexpr int kAcross = D / 32;   // warps' steps across a row
  const int block = i >> 5, in = i & 31;
  row = block / kAcross * 8 + (in & 7);
  c = block % kAcross * 4 + (in >> 3);
}

// sum[0 .. 8) = the sum over the parts of weight(i) * the eight floats at `src` and `src` +
// `rows`, `step` float4s from part to part, always in the same order.
template <typename Weight>
__device__ __forceinline__ void sum_parts(float (&sum)[8], const float4* src, int rows, size_t step,
                                          int parts, Weight&& weight) {
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < parts; i0 += 4) {
    float4 x[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i0 + i < parts) {
        x[i][0] = __ldcg(src + (size_t)(i0 + i) * step);
        x[i][1] = __ldcg(src + (size_t)(i0 + i) * step + rows);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i0 + i >= parts) break;
      const float w = weight(i0 + i);
      sum[0] = fmaf(w, x[i][0].x, sum[0]), sum[1] = fmaf(w, x[i][0].y, sum[1]);
      sum[2] = fmaf(w, x[i][0].z, sum[2]), sum[3] = fmaf(w, x[i][0].w, sum[3]);
      sum[4] = fmaf(w, x[i][1].x, sum[4]), sum[5] = fmaf(w, x[i][1].y, sum[5]);
      sum[6] = fmaf(w, x[i][1].z, sum[6]), sum[7] = fmaf(w, x[i][1].w, sum[7]);
    }
  }
}

// Eight floats times `mult` as bf16, 16 bytes.
__device__ __forceinline__ void store_bf16x8(uint16_t* dst, const float (&x)[8], float mult) {
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(pack_bf16x2(x[0] * mult, x[1] * mult), pack_bf16x2(x[2] * mult, x[3] * mult),
                 pack_bf16x2(x[4] * mult, x[5] * mult), pack_bf16x2(x[6] * mult, x[7] * mult));
}

// Shared-memory descriptor of the start of a tile, for either operand use.
// The GEMM helpers below add constant offsets to its start-address field
// (bits 0-13, address >> 4), which never carries: shared addresses stay
// below 2^18.
__device__ __forceinline__ uint64_t kmajor_tile_desc(uint32_t smem_addr) {
  return make_smem_desc_sw128(smem_addr, 16, 1024);
}

template <int D>
__device__ __forceinline__ uint64_t mnmajor_tile_desc(uint32_t smem_addr) {
  // With D = 64 there is a single slab along N and the leading offset is
  // never used; it is set to the in-slab group stride so no field can point
  // past the tile.
  return make_smem_desc_sw128(smem_addr, (D == 64) ? 1024 : kSlabBytes, 1024);
}

// S[tmem, 128 x 128 fp32] = Q K^T (or -Q K^T) for one 128-row Q tile and one
// 128-row K tile, given their K-major tile descriptors.  Both operands are
// K-major (the head dimension is contiguous): per K step of 16 elements the
// start advances
// 32 bytes inside a swizzle row, and moves to the next slab every 64
// elements.  Stride between 8-row groups (SBO) is 1024 bytes; the leading
// offset is unused for swizzled K-major operands.  Issued by one thread.
template <int D>
__device__ __forceinline__ void issue_qk_gemm(uint32_t s_tmem, uint64_t q_desc, uint64_t k_desc,
                                              bool negate = false) {
  // with `negate`, the instruction descriptor's negate-A bit gives -Q K^T
  const uint32_t idesc =
      make_idesc_bf16_f32(128, 128, false, false) | (negate ? kIdescNegateA : 0u);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = (uint64_t)(((kk >> 2) * kSlabBytes + (kk & 3) * 32) >> 4);
    mma_ss(s_tmem, q_desc + off, k_desc + off, idesc, kk > 0 ? 1u : 0u);
  }
}

// O[tmem, 128 x D fp32] (+)= P V with P [128 x 128] bf16 in tensor memory
// (row i in lane i, keys 2c and 2c+1 packed in column c) and V a
// [128 keys x D] tile used MN-major (D contiguous), given its MN-major tile
// descriptor.  Per K step of 16 keys the start advances 16 rows = 2048
// bytes; the 8-row groups along K are 1024 bytes apart (SBO); the 64-column
// slabs along N are one slab apart (LBO).  `accumulate` = false overwrites
// O.  Issued by one thread.
//
// With N > D (a multiple of 16 up to D + 64), B is [V | W]: the columns
// past D come from the 64-column atom at the descriptor's leading offset
// from V (the attention kernel's constant ones, which make those columns of
// O the row sums of P).
template <int D, int N = D>
__device__ __forceinline__ void issue_pv_gemm(uint32_t o_tmem, uint32_t p_tmem, uint64_t v_desc,
                                              bool accumulate) {
  static_assert(N % 16 == 0 && N >= D && N <= D + 64, "PV GEMM width");
  constexpr uint32_t idesc = make_idesc_bf16_f32(128, N, false, true);
#pragma unroll
  for (int kk = 0; kk < kTileRows / 16; ++kk) {
    mma_ts(o_tmem, p_tmem + kk * 8, v_desc + (uint64_t)((kk * 2048) >> 4), idesc,
           (accumulate || kk > 0) ? 1u : 0u);
  }
}

}  // namespace attnpipe
