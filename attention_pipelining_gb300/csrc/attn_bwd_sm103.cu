// attn_bwd_sm103.cu -- attention backward for sm_103a (GB300).
//
// The gradients of the forward of "PipeThreader: Software-Defined Pipelining
// for Efficient DNN Execution" (section A2, Fig. 7): with P the forward's
// softmax rows, D_i = dO_i . O_i, dP = dO V^T and dS = P o (dP - D),
//   dV = P^T dO,   dK = scale dS^T Q,   dQ = scale dS K
// (summed over the query heads that share a key/value head).  The backward
// is the subject of "GPU软件流水线与Warp Specialization优化技术解析", section
// 3.2 (Flash Attention backward on Blackwell: loads, tensor-core GEMMs and
// the elementwise work in separate warp groups).
//
// Two paths of three kernels each.  The default one (attn_bwd):
//   prep     D_i and the base-2 LSE per row, into a padded per-group
//            layout, and zeros for an fp32 dQ accumulator;
//   dK/dV    one CTA per (row group, 128 keys): over the group's query
//            blocks, S^T = K Q^T and dP^T = V dO^T on the tensor core, P^T
//            and dS^T by two elementwise warpgroups (64 queries each), then
//            dV += P^T dO and dK += dS^T Q accumulate in tensor memory, and
//            dQ^T = K^T dS^T per half block, which a fourth warpgroup reads
//            out and adds into the accumulator in L2 (kFuse);
//   convert  dq = bf16(scale * accumulator).
// The deterministic one (attn_bwd_deterministic) runs prep, dK/dV without
// dQ, and
//   dQ       one CTA per (row group, 128 query rows): over the key blocks,
//            S = Q K^T and dP = dO V^T, dS by the elementwise warpgroups (64
//            keys each), dQ += dS K in tensor memory.
// P needs no running max in the backward (the forward's LSE normalises it),
// so the elementwise work splits over columns with no exchange.
//
// Each 128 x 128 block runs as two halves of 64 columns, so the elementwise
// warps work on one half while the tensor core computes the other.
//
// 384 threads (512 with the fused dQ): warps 0-7 elementwise (warpgroup w
// takes columns 32w..32w+31 of each half, thread = TMEM lane = the tile's
// row), warp 8 tensor-core issuer and warp 9 TMA producer (warp-wide, one
// elected lane issues), warps 10-11 idle, warps 12-15 the dQ read-out.
// Every wait is bounded; a timeout raises a CTA-wide abort flag and the
// device status word records ATTN_ERR_TIMEOUT.
//
// Packed sequences (include/attn_packed.h): both paths over lists of key blocks and query
// tiles of all sequences that a plan kernel made: packed_bwd_prep_kernel, the persistent
// packed_bwd_dkdv_kernel, and packed_bwd_dq_convert_kernel or the persistent
// packed_bwd_dq_kernel.  A query tile's 128 rows are whole groups of query heads of
// consecutive tokens (row = token * R + head); the row vectors and the accumulator follow
// that order, [K/V head][token * R + head], so a tile's rows of them are contiguous.
// Behind a sequence's end the copies bring other sequences' rows: where these would meet
// a zero of P or dS in a sum over rows or keys (0 times an infinity is a NaN) the issuer
// warp clears them in shared memory first.
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <mutex>

#include "attn_internal.h"
#include "attn_tiles.cuh"
#include "kv_cache.cuh"
#include "packed_plan.cuh"
#include "ptx.cuh"

namespace attnpipe {

__device__ int g_bwd_status = 0;

namespace {

constexpr int kThreadsB = 384;
constexpr int kThreadsFused = 512;  // the dK/dV kernel with dQ: + the dQ read-out warpgroup
constexpr int kRows = 128;       // rows of a tile: keys (dK/dV kernel) or queries (dQ kernel)
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ bool warp_wait_b(uint64_t* bar, uint32_t parity,
                                            volatile int* abort_flag, uint64_t budget) {
  const bool ok = mbar_wait(bar, parity, abort_flag, budget);
  return __all_sync(kAll, ok);
}

__device__ __forceinline__ void drain_wait_b(uint64_t* bar, uint32_t parity, uint64_t budget) {
  volatile int never = 0;
  mbar_wait(bar, parity, &never, budget);
}

__device__ __forceinline__ float u2f_b(uint32_t x) { return __uint_as_float(x); }

// Adds x to the fp32 at `addr` in global memory, performed in L2 (no
// return value; relaxed, device scope).
__device__ __forceinline__ void red_add_f32(float* addr, float x) {
  asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(addr), "f"(x) : "memory");
}

// Adds `bytes` of fp32 from shared memory into global memory element by
// element (performed in L2), tracked by the issuing thread's bulk groups like
// a store.  Both addresses 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_reduce_add_f32(float* gdst, uint32_t ssrc, uint32_t bytes) {
  asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;"
               ::"l"(gdst), "r"(ssrc), "r"(bytes)
               : "memory");
}

// The work of a 128 x 128 block is done in two halves h = 0, 1 of 64
// columns, so the elementwise warpgroups work on one half while the tensor
// core runs the other half's GEMMs.

// C[tmem, 128 x 64 fp32] = A B_h^T: A a [128 x D] tile, B_h rows 64h..64h+63
// of a [128 x D] tile, both K-major (given as tile descriptors; the half's
// rows start 64 rows = 8 KB into each 128-byte-swizzled slab).
template <int D>
__device__ __forceinline__ void issue_qk_half(uint32_t c_tmem, uint64_t a_desc, uint64_t b_desc,
                                              int h) {
  constexpr uint32_t idesc = make_idesc_bf16_f32(128, 64, false, false);
  const uint64_t b_half = b_desc + (uint64_t)((h * 64 * 128) >> 4);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = (uint64_t)(((kk >> 2) * kSlabBytes + (kk & 3) * 32) >> 4);
    mma_ss(c_tmem, a_desc + off, b_half + off, idesc, kk > 0 ? 1u : 0u);
  }
}

// The same product with A in tensor memory: a [128 x D] bf16 tile copied
// there once (row i in lane i, elements 2c and 2c + 1 in column c, as the
// tensor core reads an A operand).  Only B is then read from shared memory,
// so these N = 64 products run at the tensor core's rate instead of at the
// rate shared memory can feed both operands.
template <int D>
__device__ __forceinline__ void issue_qk_half_ts(uint32_t c_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 int h) {
  constexpr uint32_t idesc = make_idesc_bf16_f32(128, 64, false, false);
  const uint64_t b_half = b_desc + (uint64_t)((h * 64 * 128) >> 4);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = (uint64_t)(((kk >> 2) * kSlabBytes + (kk & 3) * 32) >> 4);
    mma_ts(c_tmem, a_tmem + kk * 8, b_half + off, idesc, kk > 0 ? 1u : 0u);
  }
}

// Copies a [128 x D] bf16 tile from shared memory (the TMA 128-byte swizzle:
// 16-byte piece c of row r at piece c ^ (r % 8) of its 64-column slab) into
// tensor memory as an A operand (D / 2 columns from `t_col`); thread = row
// = lane of the warp's quadrant (lane_base).  Whole warp.
template <int D>
__device__ __forceinline__ void copy_tile_to_tmem(const uint8_t* tile, uint32_t t_col, int row) {
  const uint32_t base = smem_u32(tile) + (uint32_t)row * 128u;
#pragma unroll
  for (int sl = 0; sl < D / 64; ++sl) {
    uint32_t w[32];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t a, b, cc, d;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(a), "=r"(b), "=r"(cc), "=r"(d)
                   : "r"(base + (uint32_t)(sl * kSlabBytes) + 16u * (uint32_t)(c ^ (row & 7))));
      w[4 * c + 0] = a;
      w[4 * c + 1] = b;
      w[4 * c + 2] = cc;
      w[4 * c + 3] = d;
    }
    tmem_st_x32(t_col + sl * 32, w);
  }
}

// Acc[tmem, 128 x D fp32] (+)= A_h B_h: A_h [128 x 64] bf16 in tensor memory,
// two per column, written by the elementwise warpgroups (warpgroup w's 32
// elements at columns 32w .. 32w + 15 from `a_tmem`); B_h rows 64h..64h+63
// of a [128 x D] tile used MN-major (D contiguous), given its MN-major tile
// descriptor.  `accumulate` = false overwrites Acc.
template <int D>
__device__ __forceinline__ void issue_pv_half(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              int h, bool accumulate) {
  constexpr uint32_t idesc = make_idesc_bf16_f32(128, D, false, true);
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    mma_ts(d_tmem, a_tmem + (kk >> 1) * 32 + (kk & 1) * 8,
           b_desc + (uint64_t)(((4 * h + kk) * 2048) >> 4), idesc,
           (accumulate || kk > 0) ? 1u : 0u);
  }
}

// dQ^T[tmem, D x 64 fp32] = K^T dS^T_h: M = the head dimension, N = the
// half's 64 queries, K = the block's 128 keys.  A is the K tile used
// MN-major (its rows are keys, the head dimension contiguous; at D = 128
// the two 64-column slabs along M one slab apart), B the half's dS^T buffer
// used MN-major (rows are keys, 64 queries contiguous).  Per K step of 16
// keys both starts advance 16 rows = 2048 bytes.  Overwrites the
// accumulator.  Row d lands in tensor-memory lane d for D = 128; for M = 64
// rows 16 q .. 16 q + 15 land in lanes 32 q .. 32 q + 15 (measured on
// GB300 with a one-MMA probe: the other 16 lanes of each quadrant are not
// part of the result).
template <int D>
__device__ __forceinline__ void issue_dqt_half(uint32_t d_tmem, uint64_t k_desc_mn,
                                               uint64_t ds_desc_mn) {
  constexpr uint32_t idesc = make_idesc_bf16_f32(D, 64, true, true);
#pragma unroll
  for (int kk = 0; kk < kRows / 16; ++kk) {
    const uint64_t off = (uint64_t)((kk * 2048) >> 4);
    mma_ss(d_tmem, k_desc_mn + off, ds_desc_mn + off, idesc, kk > 0 ? 1u : 0u);
  }
}

template <int D>
struct BwdCfg {
  static constexpr int kTileBytes = TileShape<D>::kBytes;
  // dK/dV kernel: K, V, then a ring of (Q, dO, base-2 LSE, D) stages
  static constexpr int kQStages = (D == 128) ? 2 : 4;
  static constexpr int kVecBytes = kRows * 4;                 // one [128] fp32 vector
  static constexpr int kQStageBytes = 2 * kTileBytes + 2 * kVecBytes;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kTileBytes;
  static constexpr int kOffQRing = 2 * kTileBytes;
  // dK/dV kernel with dQ (kFuse): dS^T of one half block, [128 keys x 64
  // queries] bf16 in the 128-byte swizzle (one slab), the B operand of
  // dQ^T = K^T dS^T (MN-major)
  static constexpr int kDsBytes = kRows * 64 * 2;
  static constexpr int kOffDsT = kOffQRing + kQStages * kQStageBytes;
  // ... and at D = 64 two staging buffers for a half block's dQ partial,
  // [64 queries][64] fp32 each (the accumulator's own row layout), which one
  // bulk reduction adds into it
  static constexpr int kDqStageBytes = (D == 64) ? 64 * D * 4 : 0;
  static constexpr int kOffDqStage = kOffDsT + kDsBytes;
  static constexpr int kOffBarKV = kOffDqStage + 2 * kDqStageBytes;
  // kv_full, q_full[S], q_empty[S], sp_full[2], ps_ready[2], acc_done, drain,
  // kt_ready (K and V copied into tensor memory; D = 64), then with kFuse
  // dq_full[2], dq_free[2], ds_free
  // (and in the packed kernel kv_free, acc_free, work_full[2], work_empty[2])
  static constexpr int kNumBarsKV = 2 * kQStages + 8 + 5 + 6;
  // dK/dV kernel at D = 64: K and V as tensor-memory A operands too (D / 2
  // columns each after the two accumulators; at D = 128 there is no room)
  static constexpr bool kKVinTmem = (D == 64);
  static constexpr int kOffMiscKV = kOffBarKV + kNumBarsKV * 8;
  // packed sequences: two slots of 64 bytes for works, and a list of parts
  static constexpr int kOffWorkKV = kOffMiscKV + 16;
  static constexpr int kPartsKV = 4 * kPackedCtas / 3;   // of all CTAs
  static constexpr int kSmemKV = kOffWorkKV + 2 * 64 + kPartsKV * 4 + 1024;
  // dQ kernel: Q, dO, then a ring of (K, V) stages
  static constexpr int kKVStages = (D == 128) ? 2 : 4;
  static constexpr int kOffQ = 0;
  static constexpr int kOffDO = kTileBytes;
  static constexpr int kOffKVRing = 2 * kTileBytes;
  static constexpr int kOffBarQ = kOffKVRing + kKVStages * 2 * kTileBytes;
  // q_full, kv_full[S], kv_empty[S], sp_full[2], ds_ready[2], acc_done, drain,
  // qt_ready (Q and dO copied into tensor memory)
  // (and in the packed kernel work_full[2], work_empty[2])
  static constexpr int kNumBarsQ = 2 * kKVStages + 8 + 4;
  static constexpr int kOffMiscQ = kOffBarQ + kNumBarsQ * 8;
  // packed sequences: two slots of 64 bytes for works, and a list of parts (of both halves)
  static constexpr int kOffWorkQ = kOffMiscQ + 16;
  static constexpr int kSmemQ = kOffWorkQ + 2 * 64 + 2 * kPartsKV * 4 + 1024;
  // tensor memory: S (or S^T) [0,128), dP [128,256), accumulators after;
  // the dQ kernel keeps Q and dO as A operands (D / 2 columns each) after its
  // one accumulator.  The dK/dV kernel places the two halves as slots of
  // 128 columns instead: half h's S^T at 128 h, its dP^T at 128 h + 64 (and,
  // with kFuse, the half's dQ^T over the dP^T columns once they are read).
  static constexpr uint32_t kTmS = 0, kTmDP = 128, kTmAcc0 = 256, kTmAcc1 = 256 + D;
  static constexpr uint32_t kTmQt = 256 + D, kTmDOt = 256 + D + D / 2;
  static_assert(kTmDOt + D / 2 <= 512, "tensor memory budget of the dQ kernel");
  static constexpr uint32_t kTmKt = 256 + 2 * D, kTmVt = 256 + 2 * D + D / 2;
  static_assert(!kKVinTmem || (kTmKt < kTmVt && kTmVt + D / 2 <= 512),
                "tensor memory budget of the dK/dV kernel");
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSmemKV <= 227 * 1024 && kSmemQ <= 227 * 1024, "shared memory budget");
};

// Does query block [r0, r0 + 128) of a row group hold a row that sees a key
// of the block starting at kv0?  (Rows are head-in-group * S_q + position.)
__device__ __forceinline__ bool qblock_sees(const BwdParams& p, int r0, int kv0) {
  if (!p.causal) return true;
  const int last = min(r0 + kRows, p.R) - 1;
  if (r0 / p.S_q != last / p.S_q) return true;  // spans two heads: some row has a late position
  return last % p.S_q >= kv0;
}

// Causal grids: CTA idx -> (cost rank, row group), the costliest ranks first,
// in bands of kRankBand ranks; within a band the CTAs of one row group are
// adjacent.  The CTAs that run at once (one per SM) then cover a few row
// groups and share those groups' tiles in L2, instead of every group's (a
// rank-major order over 32 groups at 16K rows reads 256 MB of Q and dO per
// sweep, twice the L2).
constexpr int kRankBand = 16;

template <int kBand = kRankBand>
__device__ __forceinline__ void banded_rank(int idx, int n_ranks, int groups, int& rank,
                                            int& zkv) {
  const int full = n_ranks / kBand;  // whole bands
  const int per_band = groups * kBand;
  if (idx < full * per_band) {
    const int band = idx / per_band;
    const int rem = idx - band * per_band;
    zkv = rem / kBand;
    rank = band * kBand + (rem - zkv * kBand);
  } else {
    const int tail = n_ranks - full * kBand;  // ranks of the last, partial band
    const int rem = idx - full * per_band;
    zkv = rem / tail;
    rank = full * kBand + (rem - zkv * tail);
  }
}

}  // namespace

// ---------------------------------------------------------------- prep

// D_i = dO_i . O_i and LSE_i * log2(e), per row of the padded per-group
// layout [groups, Rp] (rows R..Rp-1 of a group get 0); with the fused dQ
// also zeros for the row's D fp32 accumulators.  A warp takes
// kPrepRowsPerWarp consecutive rows; a lane reads 16 bytes of O and of dO
// per row, and every load of the warp's rows is issued before any product,
// so each thread keeps several loads in flight (the kernel streams O and dO
// from HBM).
constexpr int kPrepRowsPerWarp = 8;

template <int D>
__global__ void __launch_bounds__(256) attn_bwd_prep_kernel(const BwdParams p,
                                                            const uint16_t* __restrict__ o,
                                                            const uint16_t* __restrict__ dout,
                                                            const float* __restrict__ lse) {
  constexpr int kLanesPerRow = D * 2 / 16;             // 16-byte pieces of a row
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;      // rows one warp-wide load covers
  constexpr int kLoads = kPrepRowsPerWarp / kRowsPerLoad;
  const long long row0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kPrepRowsPerWarp;
  const int lane = threadIdx.x & 31;
  const int sub = lane / kLanesPerRow;                 // row of a load
  const int piece = lane % kLanesPerRow;               // 16-byte piece within the row
  const long long total = (long long)p.groups * p.Rp;
  uint4 a[kLoads], b[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const long long row = row0 + i * kRowsPerLoad + sub;
    a[i] = make_uint4(0u, 0u, 0u, 0u);
    b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row < total) {
      const long long z = row / p.Rp;
      const int rho = (int)(row - z * p.Rp);
      if (rho < p.R) {
        const long long src = (z * p.R + rho) * D + piece * 8;
        a[i] = *reinterpret_cast<const uint4*>(o + src);
        b[i] = *reinterpret_cast<const uint4*>(dout + src);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t av[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
    const uint32_t bv[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
    float acc = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      acc += __uint_as_float(av[t] << 16) * __uint_as_float(bv[t] << 16);
      acc += __uint_as_float(av[t] & 0xffff0000u) * __uint_as_float(bv[t] & 0xffff0000u);
    }
    // sum over the row's lanes (a contiguous group of kLanesPerRow lanes)
#pragma unroll
    for (int off = kLanesPerRow / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(kAll, acc, off);
    const long long row = row0 + i * kRowsPerLoad + sub;
    if (p.dq_acc != nullptr && row < total) {
      float4* acc = reinterpret_cast<float4*>(p.dq_acc + row * D + piece * 8);
      acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
      acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (piece == 0 && row < total) {
      const long long z = row / p.Rp;
      const int rho = (int)(row - z * p.Rp);
      if (rho < p.R) {
        p.ndelta[row] = -acc;
        p.nlse2[row] = -(lse[z * p.R + rho] * 1.4426950408889634f);
      } else {
        p.ndelta[row] = 0.f;
        p.nlse2[row] = 0.f;
      }
    }
  }
}

// The same for packed sequences: rows are (token, head) in the order of O, and
// the vectors' place of a token's follows from its sequence, found by bisection.
// Bound by HBM (13 thousand tokens of 32 heads of 128, with the zeros of the accumulator:
// 385 MB of HBM traffic in 63 us, 6.1 TB/s); where there is no accumulator, by its chain of loads
// (2588 tokens of 16 heads of 64: 5.6 us).
template <int D>
__global__ void __launch_bounds__(256)
    packed_bwd_prep_kernel(const __grid_constant__ PackedBwdParams p, const uint16_t* o,
                           const uint16_t* dout, const float* lse) {
  constexpr int kLanesPerRow = D * 2 / 16;
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;
  constexpr int kLoads = kPrepRowsPerWarp / kRowsPerLoad;
  const long long row0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kPrepRowsPerWarp;
  const int lane = threadIdx.x & 31;
  const int sub = lane / kLanesPerRow, piece = lane % kLanesPerRow;
  // up to 31 sequences: the bounds by themselves, and the plan at the same time
  // (PackedPlan::early; four texts of 30 to 300 tokens, 8 heads over 2 of 64: 22.5 us, with the
  // plan first 24.2; three of 200 to 500, 8 heads of 128: 25.0 and 27.4)
  const bool first = p.cu_q != nullptr;
  int2 bounds = make_int2(0, 0);
  int q_first, q_end;
  if (first) {
    wait_for_earlier();
    allow_later();
    (void)warp_bounds(p.cu_q, p.cu_q, p.B, p.sh.T_q, p.sh.T_q, bounds);
    q_first = __shfl_sync(kAll, bounds.x, 0);
    q_end = __shfl_sync(kAll, bounds.x, p.B);
  } else {
    allow_later();
    wait_for_earlier();
    q_first = p.sh.head->q_first;
    q_end = p.sh.head->q_end;
  }
  uint4 a[kLoads], b[kLoads];
  int tok[kLoads], head[kLoads];
  float delta[kLoads];
  const long long t0 = row0 / p.H_q;
  const int h0 = (int)(row0 - t0 * p.H_q);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    long long t = t0;
    head[i] = h0 + i * kRowsPerLoad + sub;
    while (head[i] >= p.H_q) head[i] -= p.H_q, ++t;
    tok[i] = t >= q_first && t < q_end ? (int)t : -1;
    a[i] = make_uint4(0u, 0u, 0u, 0u);
    b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tok[i] >= 0) {
      a[i] = *reinterpret_cast<const uint4*>(o + t * p.o_st + head[i] * p.o_sh + piece * 8);
      b[i] = *reinterpret_cast<const uint4*>(dout + t * p.do_st + head[i] * p.do_sh + piece * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t av[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
    const uint32_t bv[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
    float acc = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      acc += __uint_as_float(av[t] << 16) * __uint_as_float(bv[t] << 16);
      acc += __uint_as_float(av[t] & 0xffff0000u) * __uint_as_float(bv[t] & 0xffff0000u);
    }
#pragma unroll
    for (int off = kLanesPerRow / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(kAll, acc, off);
    delta[i] = acc;
    if (tok[i] < 0) continue;
    const int group = p.sh.group, g = packed_over(head[i], p.sh.over_group), r = head[i] - g * group;
    if (p.dq_acc != nullptr) {
      float4* z = reinterpret_cast<float4*>(
          p.dq_acc + (((long long)g * p.sh.T_q + tok[i]) * group + r) * D + piece * 8);
      z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
      z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  // lane n < 8 has the warp's row n: its place in the vectors
  float mine = 0.f;
  int my_tok = -1, my_head = 0;
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
#pragma unroll
    for (int n = 0; n < kRowsPerLoad; ++n) {
      const float x = __shfl_sync(kAll, delta[i], n * kLanesPerRow);
      const int t = __shfl_sync(kAll, tok[i], n * kLanesPerRow);
      const int h = __shfl_sync(kAll, head[i], n * kLanesPerRow);
      if (lane == i * kRowsPerLoad + n) mine = x, my_tok = t, my_head = h;
    }
  int b0 = 0, q0 = 0;   // the last sequence that begins at or before my_tok, its first token
  if (first) {
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
      const int mid = b0 + step, begins = __shfl_sync(kAll, bounds.x, mid & 31);
      if (mid < p.B && begins <= my_tok) b0 = mid;
    }
    q0 = __shfl_sync(kAll, bounds.x, b0);
  }
  if (my_tok < 0) return;
  if (!first) {
    int b1 = p.B;   // seq_q[b0] <= my_tok < seq_q[b1]
    while (b1 - b0 > 1) {
      const int mid = (b0 + b1) >> 1;
      if (p.seq_q[mid] <= my_tok) b0 = mid;
      else b1 = mid;
    }
    q0 = p.seq_q[b0];
  }
  const int group = p.sh.group, g = packed_over(my_head, p.sh.over_group), r = my_head - g * group;
  const long long at =
      g * p.vec_stride + (long long)(packed_vec0(q0, b0) + my_tok - q0) * group + r;
  p.ndelta[at] = -mine;
  p.nlse2[at] = -(lse[(long long)my_head * p.sh.T_q + my_tok] * 1.4426950408889634f);
}

// dq = bf16(scale * dq_acc) over the tokens of the packed sequences; one thread per 8
// elements.  Bound by HBM (13 thousand tokens of 32 heads of 128: 285 MB beside what is
// still in L2, 44 us, 6.5 TB/s).
template <int D>
__global__ void __launch_bounds__(256)
    packed_bwd_dq_convert_kernel(const __grid_constant__ PackedBwdParams p) {
  constexpr int kPieces = D / 8;
  wait_for_earlier();
  // blockIdx.y: K/V head; in it (token, head in the group, piece)
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long gr = i / kPieces;
  const int piece = (int)(i % kPieces), g = (int)blockIdx.y;
  const long long t =
      p.sh.group == 1 ? gr : (long long)__umul64hi((unsigned long long)gr, p.sh.over_group64);
  const int r = (int)(gr - t * p.sh.group);
  if (t < p.sh.head->q_first || t >= p.sh.head->q_end) return;
  const long long row = (long long)g * p.sh.T_q * p.sh.group + gr;
  const float4* src = reinterpret_cast<const float4*>(p.dq_acc + row * D + piece * 8);
  const float4 a = src[0], b = src[1];
  const float sc = p.scale;
  uint4 out;
  out.x = pack_bf16x2(a.x * sc, a.y * sc);
  out.y = pack_bf16x2(a.z * sc, a.w * sc);
  out.z = pack_bf16x2(b.x * sc, b.y * sc);
  out.w = pack_bf16x2(b.z * sc, b.w * sc);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dq) + t * p.dq_st +
                            (g * p.sh.group + r) * p.dq_sh + piece * 8) = out;
}

// dq = bf16(scale * dq_acc) over the rows of every group (padding rows
// skipped); one thread per 8 elements.
template <int D>
__global__ void __launch_bounds__(256) attn_bwd_dq_convert_kernel(const BwdParams p) {
  constexpr int kPieces = D / 8;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long total = (long long)p.groups * p.R * kPieces;
  if (i >= total) return;
  const long long row = i / kPieces;   // z * R + rho
  const int piece = (int)(i - row * kPieces);
  const long long z = row / p.R;
  const long long rho = row - z * p.R;
  const float4* src = reinterpret_cast<const float4*>(p.dq_acc + (z * p.Rp + rho) * D + piece * 8);
  const float4 a = src[0], b = src[1];
  const float sc = p.scale;
  uint4 out;
  out.x = pack_bf16x2(a.x * sc, a.y * sc);
  out.y = pack_bf16x2(a.z * sc, a.w * sc);
  out.z = pack_bf16x2(b.x * sc, b.y * sc);
  out.w = pack_bf16x2(b.z * sc, b.w * sc);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dq) + row * D + piece * 8) = out;
}

// ---------------------------------------------------------------- dK, dV

// kFuse: dQ too.  Per half block the tensor core also computes
// dQ^T = K^T dS^T (dS^T from a shared buffer the elementwise warps write)
// into the half's dP^T columns, and warps 12-15 read it out and add it into
// the fp32 accumulator p.dq_acc in L2 (red.global.add); dS^T for dK then
// sits in tensor memory next to P^T.  512 threads.
template <int D, bool kFuse>
__global__ void __launch_bounds__(kFuse ? kThreadsFused : kThreadsB, 1)
    attn_bwd_dkdv_kernel(const __grid_constant__ BwdParams p) {
  using C = BwdCfg<D>;
  extern __shared__ uint8_t smem_raw_b[];
  uint8_t* smem = align_smem_1024(smem_raw_b);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBarKV);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;
  uint64_t* q_empty = q_full + C::kQStages;
  uint64_t* sp_full = q_empty + C::kQStages;   // [half]: S^T, dP^T of the half computed
  uint64_t* ps_ready = sp_full + 2;            // [half]: P^T, dS^T of the half stored
  uint64_t* acc_done = sp_full + 4;
  uint64_t* drain = sp_full + 5;
  uint64_t* kt_ready = sp_full + 6;            // K and V copied into tensor memory (D = 64)
  uint64_t* dq_full = sp_full + 7;             // [half]: dQ^T of the half computed (kFuse)
  uint64_t* dq_free = sp_full + 9;             // [half]: dQ^T of the half read out (kFuse)
  uint64_t* ds_free = sp_full + 11;            // the GEMMs reading the dS^T buffer are done
  uint8_t* sDsT = smem + C::kOffDsT;
  uint32_t* sTmemBase = reinterpret_cast<uint32_t*>(smem + C::kOffMiscKV);
  volatile int* sAbort = reinterpret_cast<volatile int*>(smem + C::kOffMiscKV + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t budget = p.timeout_ns;

  // CTA -> (key block, row group): with the causal mask the first key
  // blocks carry the most query blocks, so they go first (in bands, see
  // banded_rank); without it the blocks of one group are adjacent (they
  // share their Q and dO tiles in L2)
  const int n_kvb = (p.S_kv + kRows - 1) / kRows;
  int kvb, zkv;
  if (p.causal) {
    banded_rank((int)blockIdx.x, n_kvb, p.groups, kvb, zkv);
  } else {
    zkv = blockIdx.x / n_kvb;
    kvb = blockIdx.x - zkv * n_kvb;
  }
  const int kv0 = kvb * kRows;              // first key of the block
  const int n_qb = (p.R + kRows - 1) / kRows;
  // the order every role walks the query blocks in: with kFuse and no mask
  // rotated by the key block, so the CTAs running at once add into
  // different dQ rows (with the causal mask each key block starts at its own
  // diagonal anyway)
  const int rot = (kFuse && !p.causal) ? kvb % n_qb : 0;
  auto qb_at = [&](int i) { return i + rot < n_qb ? i + rot : i + rot - n_qb; };
  // The query blocks with work (items n = 0 .. n_work - 1), walked by every
  // role in the same order.  With the causal mask and S_q a multiple of 128
  // no block spans two heads, and block pb of a head sees keys kv0 .. when
  // its last position pb * 128 + 127 >= kv0, i.e. pb >= kvb: the items are
  // those blocks of each head in turn, found without a scan (a scan's
  // division per skipped block cost a short CTA tens of microseconds).
  // Otherwise (a ragged S_q) the blocks are scanned with qblock_sees.
  const bool by_head = p.causal && (p.S_q % kRows == 0);
  const int nqh = by_head ? p.S_q / kRows : 1;             // position blocks per head
  const int per_head = by_head ? (nqh > kvb ? nqh - kvb : 0) : 0;
  int n_work = 0;
  if (!p.causal) {
    n_work = n_qb;
  } else if (by_head) {
    n_work = (p.R / p.S_q) * per_head;
  } else {
    for (int qb = 0; qb < n_qb; ++qb) n_work += qblock_sees(p, qb * kRows, kv0) ? 1 : 0;
  }
  // first row of item n's query block; `cursor` is the caller's scan
  // position (the ragged causal case only; items are asked for in order)
  auto item_r0 = [&](int n, int& cursor) -> int {
    if (!p.causal) return qb_at(n) * kRows;
    if (by_head) {
      const int h = n / per_head;
      return (h * nqh + kvb + (n - h * per_head)) * kRows;
    }
    while (cursor < n_qb - 1 && !qblock_sees(p, cursor * kRows, kv0)) ++cursor;
    return (cursor++) * kRows;
  };

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < C::kQStages; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sp_full[h], 1);
      mbar_init(&ps_ready[h], 2 * 128);
    }
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    mbar_init(kt_ready, 2 * 128);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&dq_full[h], 1);
      mbar_init(&dq_free[h], 128);
    }
    mbar_init(ds_free, 1);
    *sAbort = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(sTmemBase, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *sTmemBase;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  auto stage_q = [&](int s) { return smem + C::kOffQRing + s * C::kQStageBytes; };
  auto stage_do = [&](int s) { return stage_q(s) + C::kTileBytes; };
  auto stage_lse = [&](int s) {
    return reinterpret_cast<float*>(stage_q(s) + 2 * C::kTileBytes);
  };
  auto stage_delta = [&](int s) {
    return reinterpret_cast<float*>(stage_q(s) + 2 * C::kTileBytes + C::kVecBytes);
  };

  if (warp < 8) {
    // -------------------------------------------------------- elementwise
    // half h of a block is queries 64h .. 64h + 63; warpgroup w takes
    // queries 64h + 32w .. 64h + 32w + 31 of it
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;          // key row within the block
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int key = kv0 + r;
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    bool ok = true;
    if constexpr (C::kKVinTmem) {
      // K (warpgroup 0) and V (warpgroup 1) into tensor memory, the A
      // operands of every S^T and dP^T product of this CTA
      if (n_work > 0) {
        ok = warp_wait_b(kv_full, 0, sAbort, budget);
        if (ok) {
          copy_tile_to_tmem<D>(w == 0 ? sK : sV, tmem + lane_base + (w == 0 ? C::kTmKt : C::kTmVt), r);
          tmem_st_wait();
          tc_fence_before_sync();
          mbar_arrive(kt_ready);
        }
      }
    }
    int cursor = 0;
    for (int n = 0; n < n_work && ok; ++n) {
      const int r0 = item_r0(n, cursor);
      const int s = n % C::kQStages;
      // masking: rows past R, keys past S_kv, and (causal) keys after a row's
      // position; a block needs none when every row sees every key
      bool masked = (r0 + kRows > p.R) || (kv0 + kRows > p.S_kv);
      int base_pos = 0;
      if (p.causal) {
        base_pos = r0 % p.S_q;
        const bool one_head = (base_pos + kRows <= p.S_q);
        masked = masked || !(one_head && base_pos >= kv0 + kRows - 1);
      }
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (!warp_wait_b(&sp_full[h], n & 1, sAbort, budget)) { ok = false; break; }
        // the stage's LSE and D vectors arrived with its tiles: observe that
        // phase here too before reading them
        if (h == 0 && !warp_wait_b(&q_full[s], (n / C::kQStages) & 1, sAbort, budget)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const int col0 = 64 * h + 32 * w;            // first query of this thread's slice
        const uint32_t cS = 128 * h + 32 * w;        // its S^T columns (dP^T: + 64)
        uint32_t sv[32], dp[32];
        tmem_ld_x32(tmem + lane_base + cS, sv);
        tmem_ld_x32(tmem + lane_base + cS + 64, dp);
        const float4* lse4 = reinterpret_cast<const float4*>(stage_lse(s) + col0);
        const float4* dl4 = reinterpret_cast<const float4*>(stage_delta(s) + col0);
        tmem_ld_wait();
        reg_after_wait(sv);
        reg_after_wait(dp);
        uint32_t pk[16], dk[16];
        // The masked and unmasked bodies are separate code paths, so the
        // common (unmasked) one carries no per-element mask arithmetic.
        auto body = [&](auto masked_tag) {
          constexpr bool kMasked = decltype(masked_tag)::value;
#pragma unroll
          for (int i4 = 0; i4 < 8; ++i4) {
            const float4 l4 = lse4[i4];              // -LSE * log2(e) of 4 queries
            const float4 d4 = dl4[i4];               // -D of the same queries
            const int c = 4 * i4;                    // first element of the four
            // x = s * scale * log2(e) - LSE * log2(e), two lanes per instruction
            float x[4];
            f2_unpack(f2_fma(f2_pack(u2f_b(sv[c]), u2f_b(sv[c + 1])), sl2x2, f2_pack(l4.x, l4.y)),
                      x[0], x[1]);
            f2_unpack(f2_fma(f2_pack(u2f_b(sv[c + 2]), u2f_b(sv[c + 3])), sl2x2,
                             f2_pack(l4.z, l4.w)), x[2], x[3]);
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float pv = ex2_approx(x[e]);
              if constexpr (kMasked) {
                const int rho = r0 + col0 + c + e;
                bool vis = (rho < p.R) && (key < p.S_kv);
                if (p.causal) {
                  int pos;
                  if (p.S_q >= kRows) {
                    pos = base_pos + col0 + c + e;
                    if (pos >= p.S_q) pos -= p.S_q;
                  } else {
                    pos = rho % p.S_q;
                  }
                  vis = vis && (key <= pos);
                }
                pv = vis ? pv : 0.f;
              }
              pr[e] = pv;
            }
            // dS = P (dP - D)
            const uint64_t ds01 = f2_mul(f2_pack(pr[0], pr[1]),
                                         f2_add(f2_pack(u2f_b(dp[c]), u2f_b(dp[c + 1])),
                                                f2_pack(d4.x, d4.y)));
            const uint64_t ds23 = f2_mul(f2_pack(pr[2], pr[3]),
                                         f2_add(f2_pack(u2f_b(dp[c + 2]), u2f_b(dp[c + 3])),
                                                f2_pack(d4.z, d4.w)));
            float d0, d1, d2, d3;
            f2_unpack(ds01, d0, d1);
            f2_unpack(ds23, d2, d3);
            pk[2 * i4] = pack_bf16x2(pr[0], pr[1]);
            pk[2 * i4 + 1] = pack_bf16x2(pr[2], pr[3]);
            dk[2 * i4] = pack_bf16x2(d0, d1);
            dk[2 * i4 + 1] = pack_bf16x2(d2, d3);
          }
        };
        if (masked)
          body(std::true_type{});
        else
          body(std::false_type{});
        // P^T of the slice: 16 columns from its S^T columns (this
        // warpgroup's own, already read)
        tmem_st_x16(tmem + lane_base + cS, pk);
        if constexpr (kFuse) {
          // dS^T of the slice into the shared buffer (row = key, this
          // warpgroup's 32 queries = 16-byte pieces 4w .. 4w + 3 of the
          // swizzled row), once the previous half's GEMMs have read it
          const int nh = 2 * n + h;
          if (nh > 0 && !warp_wait_b(ds_free, (nh - 1) & 1, sAbort, budget)) {
            ok = false;
            break;
          }
          const uint32_t row = smem_u32(sDsT) + (uint32_t)r * 128u;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st_shared_v4(row + 16u * (uint32_t)((4 * w + j) ^ (r & 7)), dk[4 * j], dk[4 * j + 1],
                         dk[4 * j + 2], dk[4 * j + 3]);
          fence_proxy_async_smem();  // the tensor core reads it through the async proxy
          // and into the slice's own S^T columns 16-31 (dK's A operand): the
          // half's dP^T columns take dQ^T
          tmem_st_x16(tmem + lane_base + cS + 16, dk);
        } else {
          // dS^T over the slice's dP^T columns, likewise
          tmem_st_x16(tmem + lane_base + cS + 64, dk);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        if (!(w == 0 && h == 0 && n == p.fault_drop_item)) mbar_arrive(&ps_ready[h]);
      }
    }
    // ---------------------------------------------------------- epilogue
    // warpgroup w writes columns [D/2 w, D/2 (w + 1)) of dV and dK
    bool have_acc = ok && n_work > 0;
    if (have_acc) {
      if (!warp_wait_b(acc_done, 0, sAbort, budget)) { ok = false; have_acc = false; }
      tc_fence_after_sync();
    }
    const bool row_ok = key < p.S_kv;
    uint16_t* dk_row = static_cast<uint16_t*>(p.dk) + ((size_t)zkv * p.S_kv + key) * D;
    uint16_t* dv_row = static_cast<uint16_t*>(p.dv) + ((size_t)zkv * p.S_kv + key) * D;
#pragma unroll
    for (int which = 0; which < 2; ++which) {  // 0: dV, 1: dK
      uint16_t* dst = which ? dk_row : dv_row;
      const float mult = which ? p.scale : 1.f;
      const uint32_t acc = tmem + lane_base + (which ? C::kTmAcc1 : C::kTmAcc0) + (D / 2) * w;
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch) {
        uint32_t v[32];
        if (have_acc) {
          tmem_ld_x32(acc + ch * 32, v);
          tmem_ld_wait();
          reg_after_wait(v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;  // no query sees these keys
        }
        if (row_ok && ok) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + (D / 2) * w + ch * 32);
#pragma unroll
          for (int qd = 0; qd < 4; ++qd) {
            uint4 val;
            val.x = pack_bf16x2(u2f_b(v[qd * 8 + 0]) * mult, u2f_b(v[qd * 8 + 1]) * mult);
            val.y = pack_bf16x2(u2f_b(v[qd * 8 + 2]) * mult, u2f_b(v[qd * 8 + 3]) * mult);
            val.z = pack_bf16x2(u2f_b(v[qd * 8 + 4]) * mult, u2f_b(v[qd * 8 + 5]) * mult);
            val.w = pack_bf16x2(u2f_b(v[qd * 8 + 6]) * mult, u2f_b(v[qd * 8 + 7]) * mult);
            d4[qd] = val;
          }
        }
      }
    }
  } else if (warp == 8) {
    // -------------------------------------------------------- tensor-core issuer
    const bool leader = elect_one();
    const uint64_t dK = kmajor_tile_desc(smem_u32(sK));
    const uint64_t dV = kmajor_tile_desc(smem_u32(sV));
    // half h's slot: S^T (then P^T) at 128 h, dP^T (then dQ^T) at 128 h + 64
    const uint32_t tS = tmem, tDP = tmem + 64;
    const uint32_t tdV = tmem + C::kTmAcc0, tdK = tmem + C::kTmAcc1;
    bool ok = n_work > 0 &&
              warp_wait_b(C::kKVinTmem ? kt_ready : kv_full, 0, sAbort, budget);
    // S^T and dP^T of half h of work item n (its Q / dO stage is loaded);
    // at D = 64 K and V are read from tensor memory
    auto issue_sp = [&](int n, int h) {
      const int s = n % C::kQStages;
      if (leader) {
        if constexpr (C::kKVinTmem) {
          issue_qk_half_ts<D>(tS + 128 * h, tmem + C::kTmKt, kmajor_tile_desc(smem_u32(stage_q(s))), h);
          issue_qk_half_ts<D>(tDP + 128 * h, tmem + C::kTmVt, kmajor_tile_desc(smem_u32(stage_do(s))), h);
        } else {
          issue_qk_half<D>(tS + 128 * h, dK, kmajor_tile_desc(smem_u32(stage_q(s))), h);
          issue_qk_half<D>(tDP + 128 * h, dV, kmajor_tile_desc(smem_u32(stage_do(s))), h);
        }
        tc_commit(&sp_full[h]);
      }
    };
    if (ok && warp_wait_b(&q_full[0], 0, sAbort, budget)) {
      tc_fence_after_sync();
      issue_sp(0, 0);
      issue_sp(0, 1);
    } else {
      ok = false;
    }
    for (int n = 0; n < n_work && ok; ++n) {
      const int s = n % C::kQStages;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (!warp_wait_b(&ps_ready[h], n & 1, sAbort, budget)) { ok = false; break; }
        tc_fence_after_sync();
        if (leader) {
          if constexpr (kFuse) {
            // dQ^T = K^T dS^T first, so its read-out overlaps the next two;
            // it is the only reader of the dS^T buffer
            issue_dqt_half<D>(tDP + 128 * h, mnmajor_tile_desc<D>(smem_u32(sK)),
                              mnmajor_tile_desc<64>(smem_u32(sDsT)));
            tc_commit(&dq_full[h]);
            tc_commit(ds_free);
          }
          // dV += P^T dO and dK += dS^T Q over this half's 64 queries; with
          // kFuse dS^T sits in the S^T columns next to P^T (columns 16-31 of
          // each warpgroup's 32), otherwise over the dP^T columns
          issue_pv_half<D>(tdV, tS + 128 * h, mnmajor_tile_desc<D>(smem_u32(stage_do(s))), h,
                           n > 0 || h > 0);
          issue_pv_half<D>(tdK, kFuse ? tS + 128 * h + 16 : tDP + 128 * h,
                           mnmajor_tile_desc<D>(smem_u32(stage_q(s))), h, n > 0 || h > 0);
          if (h == 1) tc_commit(&q_empty[s]);  // both halves read: the stage is free
        }
        // the next item's half h overwrites what these GEMMs read: issued
        // after them by the same thread, it runs after them
        if (n + 1 < n_work) {
          if (h == 0) {
            if (!warp_wait_b(&q_full[(n + 1) % C::kQStages], ((n + 1) / C::kQStages) & 1,
                             sAbort, budget)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
          }
          if constexpr (kFuse) {
            // ... and over this half's dQ^T once it has been read out
            if (!warp_wait_b(&dq_free[h], n & 1, sAbort, budget)) { ok = false; break; }
            tc_fence_after_sync();
          }
          issue_sp(n + 1, h);
        }
      }
    }
    if (ok && leader) tc_commit(acc_done);
    if (leader) {
      tc_commit(drain);
      drain_wait_b(drain, 0, budget);
    }
    __syncwarp();
  } else if (warp == 9) {
    // -------------------------------------------------------- TMA producer
    const bool leader = elect_one();
    const uint64_t pol_kv = l2_policy_evict_first();
    const uint64_t pol_q = l2_policy_evict_last();
    int issued = 0;
    bool ok = n_work > 0;
    if (ok && leader) {
      mbar_arrive_expect_tx(kv_full, 2 * C::kTileBytes);
      tma_load_tile<D>(sK, &p.tm_k, kv_full, kv0, zkv, pol_kv);
      tma_load_tile<D>(sV, &p.tm_v, kv_full, kv0, zkv, pol_kv);
    }
    int cursor = 0;
    for (int n = 0; n < n_work && ok; ++n) {
      const int r0 = item_r0(n, cursor);
      const int s = issued % C::kQStages;
      const int round = issued / C::kQStages;
      if (round > 0 && !warp_wait_b(&q_empty[s], (round - 1) & 1, sAbort, budget)) {
        ok = false;
        break;
      }
      if (leader) {
        mbar_arrive_expect_tx(&q_full[s], 2 * C::kTileBytes + 2 * C::kVecBytes);
        tma_load_tile<D>(stage_q(s), &p.tm_q, &q_full[s], r0, zkv, pol_q);
        tma_load_tile<D>(stage_do(s), &p.tm_do, &q_full[s], r0, zkv, pol_q);
        const size_t vo = (size_t)zkv * p.Rp + r0;
        bulk_load(stage_lse(s), p.nlse2 + vo, C::kVecBytes, &q_full[s]);
        bulk_load(stage_delta(s), p.ndelta + vo, C::kVecBytes, &q_full[s]);
      }
      ++issued;
    }
    if (leader) {
      if (n_work > 0) drain_wait_b(kv_full, 0, budget);
      const int first = issued > C::kQStages ? issued - C::kQStages : 0;
      for (int t = first; t < issued; ++t)
        drain_wait_b(&q_full[t % C::kQStages], (t / C::kQStages) & 1, budget);
    }
    __syncwarp();
  } else if (kFuse && warp >= 12) {
    // -------------------------------------------------------- dQ read-out
    // thread = TMEM lane = head dimension d (D = 64: lanes 0-15 of each
    // quadrant, d = 16 q + lane); per half block it takes the 64 queries'
    // dQ^T values of its d and adds them into rows r0 + 64 h + j of the
    // group's fp32 accumulator (a warp's lanes cover 128 or 64 contiguous
    // bytes of a row)
    const bool has_d = (D == 128) || lane < 16;
    const int d = (D == 128) ? (warp & 3) * 32 + lane : (warp & 3) * 16 + (lane & 15);
    // D = 64: a warp's red would carry 64 bytes only, and the L2 takes
    // requests at a bounded rate whatever their size; instead the half's
    // values go to a staging buffer and one thread adds all 16 KB with a
    // bulk reduction (one bulk group per half block; two buffers)
    float* sStage = reinterpret_cast<float*>(smem + C::kOffDqStage);
    int nh = 0;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    bool ok = true;
    int cursor = 0;
    for (int n = 0; n < n_work && ok; ++n) {
      const int r0 = item_r0(n, cursor);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if constexpr (D == 64) {
          // the bulk reduction that read this half's staging buffer two
          // halves ago is done (one bulk group per half)
          if (threadIdx.x == 12 * 32) tma_store_wait_read<1>();
        }
        const bool got = warp_wait_b(&dq_full[h], n & 1, sAbort, budget);
        if constexpr (D == 64) {
          // the four warps agree (they meet at named barriers below, which
          // no warp may skip); this also orders the buffer's reuse
          if (barrier_or(1, 128, !got)) { ok = false; break; }
        } else {
          if (!got) { ok = false; break; }
        }
        tc_fence_after_sync();
        uint32_t v0[32], v1[32];
        tmem_ld_x32(tmem + lane_base + 128 * h + 64, v0);
        tmem_ld_x32(tmem + lane_base + 128 * h + 96, v1);
        tmem_ld_wait();
        reg_after_wait(v0);
        reg_after_wait(v1);
        tc_fence_before_sync();
        mbar_arrive(&dq_free[h]);            // the columns may be overwritten
        const int q0 = r0 + 64 * h;
        if constexpr (D == 128) {
          const int rows = p.R - q0;           // rows past R are padding: skipped
          float* dst = p.dq_acc + ((size_t)zkv * p.Rp + q0) * D + d;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < rows) red_add_f32(dst + (size_t)j * D, u2f_b(v0[j]));
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (32 + j < rows) red_add_f32(dst + (size_t)(32 + j) * D, u2f_b(v1[j]));
        } else {
          float* stg = sStage + (nh & 1) * 64 * D;
          if (has_d) {
#pragma unroll
            for (int j = 0; j < 32; ++j) stg[j * D + d] = u2f_b(v0[j]);
#pragma unroll
            for (int j = 0; j < 32; ++j) stg[(32 + j) * D + d] = u2f_b(v1[j]);
          }
          fence_proxy_async_smem();            // the bulk copy reads through the async proxy
          named_barrier_sync(1, 128);
          if (threadIdx.x == 12 * 32) {
            const int rows = min(64, p.R - q0);  // rows past R are padding: skipped
            if (rows > 0)
              bulk_reduce_add_f32(p.dq_acc + ((size_t)zkv * p.Rp + q0) * D, smem_u32(stg),
                                  (uint32_t)rows * D * 4);
            tma_store_commit();                // one group per half, possibly empty
          }
          ++nh;
        }
      }
    }
    // every bulk reduction has read its buffer and reached global memory
    if (D == 64 && threadIdx.x == 12 * 32) tma_store_wait_all();
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 8) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0 && *sAbort) atomicCAS(&g_bwd_status, 0, (int)ATTN_ERR_TIMEOUT);
}

// ---------------------------------------------------------------- dK, dV, packed

// One work item of the kernel below: a block of keys and a K/V head.
struct PackedWork {
  int valid;
  int n_keys, head, tok_k;               // keys of the block, K/V head, first key token
  int tok_q, q_len, vec0, shift;         // as in PackedKeys, of the block
  int first, n_work, tiles;              // its query tiles
  int part, slot, parts;
  int unused[2];
};

// The blocks of a group come one K/V head after the other; any entry of the group says
// what the group is, so one load is enough.
__device__ __forceinline__ PackedWork packed_work(const PackedBwdParams& p, int entries, int idx) {
  PackedWork x;
  const int at = idx / p.H_kv;
  x.valid = at < entries;
  if (!x.valid) return x;
  const int4* src = reinterpret_cast<const int4*>(p.sh.keys + at);
  const int4 a = src[0], b = src[1], c = src[2], d = src[3];   // in PackedKeys' order
  const int size = b.z;
  const int in_group = idx - (at - b.w) * p.H_kv;              // (head, block)
  x.head = in_group / size;
  const int t = in_group - x.head * size;
  x.tok_k = a.x + t * kRows;
  x.n_keys = min(a.y - t * kRows, kRows);
  x.tok_q = a.z;
  x.q_len = a.w;
  x.vec0 = b.x;
  x.shift = b.y + t * kRows;
  x.tiles = c.x;
  x.part = c.y;
  x.slot = c.z;
  x.parts = c.w;
  if (c.w > 1) {
    x.first = d.x;
    x.n_work = d.y;
  } else if (p.causal) {
    x.first = min(packed_over(max(x.shift, 0), p.sh.over_positions), x.tiles);
    x.n_work = x.tiles - x.first;
  } else {   // each block begins elsewhere, so that those that run at once add to different rows
    x.first = x.tiles > 0 ? (d.x + t) % x.tiles : 0;
    x.n_work = x.tiles;
  }
  return x;
}

// attn_bwd_dkdv_kernel over packed sequences, persistent: with short sequences a block of
// keys has a few query tiles only, and a thread block of its own for each spent most of
// its time starting and ending (16 x 16 heads of 64, queries of 20 to 1000 tokens over
// keys of 64 to 2304: 77 us, so 56).  The producer warp takes the next work from a counter
// (the costliest come first), tells the other roles what it is in one of two slots of
// shared memory, and loads ahead as far as the ring and the K and V buffers allow, while
// the work before is finished and its dK and dV are written.  The roles, the products and
// their hand-offs are attn_bwd_dkdv_kernel's, their phases counted on from work to work;
// beside them
//   kv_free    the work's products have read K and V (shared memory)
//   acc_free   dV and dK have been read out of tensor memory
//   work_full, work_empty [slot]
// Which thread block does which work differs from run to run; no result depends on it
// (with kFuse the order of the additions to dQ does).
//
// Bound by the chain of hand-offs between the products and the elementwise warps: 12 documents
// of 100 to 4096 tokens, 32 heads over 8 of 128, causal, 604 GFLOP in 576 us (1050 TFLOP/s;
// the tensor pipe is busy in 47 % of the cycles: masked halves of diagonal blocks and tiles
// that a sequence does not fill are computed too).  With the next work asked for when the
// one before begins, not when it ends, that call took 773 us instead of 716 (694 now):
// works were bound to CTAs that were long busy.
template <int D, bool kFuse>
__global__ void __launch_bounds__(kFuse ? kThreadsFused : kThreadsB, 1)
    packed_bwd_dkdv_kernel(const __grid_constant__ PackedBwdParams p) {
  using C = BwdCfg<D>;
  extern __shared__ uint8_t smem_raw_b[];
  uint8_t* smem = align_smem_1024(smem_raw_b);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBarKV);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;
  uint64_t* q_empty = q_full + C::kQStages;
  uint64_t* sp_full = q_empty + C::kQStages;
  uint64_t* ps_ready = sp_full + 2;
  uint64_t* acc_done = sp_full + 4;
  uint64_t* drain = sp_full + 5;
  uint64_t* kt_ready = sp_full + 6;
  uint64_t* dq_full = sp_full + 7;
  uint64_t* dq_free = sp_full + 9;
  uint64_t* ds_free = sp_full + 11;
  uint64_t* kv_free = sp_full + 12;
  uint64_t* acc_free = sp_full + 13;
  uint64_t* work_full = sp_full + 14;
  uint64_t* work_empty = sp_full + 16;
  uint8_t* sDsT = smem + C::kOffDsT;
  uint32_t* sTmemBase = reinterpret_cast<uint32_t*>(smem + C::kOffMiscKV);
  volatile int* sAbort = reinterpret_cast<volatile int*>(smem + C::kOffMiscKV + 4);
  volatile int* sFlag = reinterpret_cast<volatile int*>(smem + C::kOffMiscKV + 8);
  volatile int* sNumParts = reinterpret_cast<volatile int*>(smem + C::kOffMiscKV + 12);
  PackedWork* sWork = reinterpret_cast<PackedWork*>(smem + C::kOffWorkKV);
  int* sParts = reinterpret_cast<int*>(smem + C::kOffWorkKV + 2 * sizeof(PackedWork));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t budget = p.timeout_ns;
  const int group = p.sh.group, positions = p.sh.positions;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < C::kQStages; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sp_full[h], 1);
      mbar_init(&ps_ready[h], 2 * 128);
      mbar_init(&dq_full[h], 1);
      mbar_init(&dq_free[h], 128);
      mbar_init(&work_full[h], 1);
      mbar_init(&work_empty[h], 9 + (kFuse ? 4 : 0));   // warps 0-8, 12-15
    }
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    mbar_init(kt_ready, 2 * 128);
    mbar_init(ds_free, 1);
    mbar_init(kv_free, 1);
    mbar_init(acc_free, 2 * 128);
    *sAbort = 0;
    *sNumParts = 0;
    fence_mbar_init();
  }
  // the spare rows of the Q and dO tiles, which no copy writes
  if (group * positions < kRows && warp < 2 * C::kQStages)
    clear_rows<D>(smem + C::kOffQRing + (warp >> 1) * C::kQStageBytes + (warp & 1) * C::kTileBytes,
                  group * positions);
  if (warp == 8) {
    tmem_alloc(sTmemBase, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *sTmemBase;
  wait_for_earlier();
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  auto stage_q = [&](int s) { return smem + C::kOffQRing + s * C::kQStageBytes; };
  auto stage_do = [&](int s) { return stage_q(s) + C::kTileBytes; };
  auto stage_lse = [&](int s) {
    return reinterpret_cast<float*>(stage_q(s) + 2 * C::kTileBytes);
  };
  auto stage_delta = [&](int s) {
    return reinterpret_cast<float*>(stage_q(s) + 2 * C::kTileBytes + C::kVecBytes);
  };
  // the w-th work of this CTA, once it is known; nullptr behind the last (or when a wait
  // ran out)
  auto work_at = [&](int w) -> const PackedWork* {
    if (!warp_wait_b(&work_full[w & 1], (w >> 1) & 1, sAbort, budget)) return nullptr;
    const PackedWork* x = sWork + (w & 1);
    return x->valid ? x : nullptr;
  };
  auto work_done = [&](int w) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&work_empty[w & 1]);
  };
  // first query position of the n-th tile of a work
  auto tile_r0 = [&](int first, int tiles, int n) {
    const int t = first + n;
    return (t < tiles ? t : t - tiles) * positions;
  };

  if (warp < 8) {
    // -------------------------------------------------------- elementwise
    const int wg = warp >> 2;
    const int r = (warp & 3) * 32 + lane;          // key row within the block
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    int item = 0;                                  // query tiles so far
    uint32_t wk = 0;                               // works with any so far
    bool ok = true, copied = false;
    // K (warpgroup 0) and V (warpgroup 1) of the n-th work with any into tensor memory; the
    // products of the work before, which read them there, are done (acc_done below)
    auto copy_keys = [&](uint32_t n) {
      if (!warp_wait_b(kv_full, n & 1, sAbort, budget)) return false;
      copy_tile_to_tmem<D>(wg == 0 ? sK : sV,
                           tmem + lane_base + (wg == 0 ? C::kTmKt : C::kTmVt), r);
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(kt_ready);
      return true;
    };
    for (int w = 0; ok; ++w) {
      const PackedWork* x = work_at(w);
      if (!x) break;
      const int n_work = x->n_work, n_keys = x->n_keys;
      if constexpr (C::kKVinTmem) {
        if (n_work > 0 && !copied && !copy_keys(wk)) break;
        copied = false;
      }
      const int first = x->first, tiles = x->tiles, q_len = x->q_len, shift = x->shift;
      for (int n = 0; n < n_work && ok; ++n, ++item) {
        const int r0 = tile_r0(first, tiles, n);
        const int s = item % C::kQStages;
        // the tile's rows that see this thread's key; no masking where every row sees
        // every key
        int row_lo = 0, row_hi = min(q_len - r0, positions) * group;
        const bool masked =
            row_hi < kRows || n_keys < kRows || (p.causal && r0 < shift + kRows - 1);
        if (p.causal) row_lo = min(max(r + shift - r0, 0), kRows) * group;
        if (r >= n_keys) row_hi = 0;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (!warp_wait_b(&sp_full[h], item & 1, sAbort, budget)) { ok = false; break; }
          if (h == 0 && !warp_wait_b(&q_full[s], (item / C::kQStages) & 1, sAbort, budget)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const int col0 = 64 * h + 32 * wg;
          const uint32_t cS = 128 * h + 32 * wg;
          uint32_t sv[32], dp[32];
          tmem_ld_x32(tmem + lane_base + cS, sv);
          tmem_ld_x32(tmem + lane_base + cS + 64, dp);
          const float4* lse4 = reinterpret_cast<const float4*>(stage_lse(s) + col0);
          const float4* dl4 = reinterpret_cast<const float4*>(stage_delta(s) + col0);
          tmem_ld_wait();
          reg_after_wait(sv);
          reg_after_wait(dp);
          uint32_t pk[16], dk[16];
          auto body = [&](auto masked_tag) {
            constexpr bool kMasked = decltype(masked_tag)::value;
#pragma unroll
            for (int i4 = 0; i4 < 8; ++i4) {
              const float4 l4 = lse4[i4];              // -LSE * log2(e) of 4 queries
              const float4 d4 = dl4[i4];               // -D of the same queries
              const int c = 4 * i4;
              float e[4];
              f2_unpack(f2_fma(f2_pack(u2f_b(sv[c]), u2f_b(sv[c + 1])), sl2x2,
                               f2_pack(l4.x, l4.y)), e[0], e[1]);
              f2_unpack(f2_fma(f2_pack(u2f_b(sv[c + 2]), u2f_b(sv[c + 3])), sl2x2,
                               f2_pack(l4.z, l4.w)), e[2], e[3]);
              bool sees[4];
              float pr[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                sees[i] = !kMasked || (col0 + c + i >= row_lo && col0 + c + i < row_hi);
                pr[i] = sees[i] ? ex2_approx(e[i]) : 0.f;
              }
              // dS = P (dP - D)
              float ds[4];
              f2_unpack(f2_mul(f2_pack(pr[0], pr[1]),
                               f2_add(f2_pack(u2f_b(dp[c]), u2f_b(dp[c + 1])),
                                      f2_pack(d4.x, d4.y))), ds[0], ds[1]);
              f2_unpack(f2_mul(f2_pack(pr[2], pr[3]),
                               f2_add(f2_pack(u2f_b(dp[c + 2]), u2f_b(dp[c + 3])),
                                      f2_pack(d4.z, d4.w))), ds[2], ds[3]);
              // (what a masked dP or D holds may be another sequence's infinity)
#pragma unroll
              for (int i = 0; i < 4; ++i) ds[i] = sees[i] ? ds[i] : 0.f;
              pk[2 * i4] = pack_bf16x2(pr[0], pr[1]);
              pk[2 * i4 + 1] = pack_bf16x2(pr[2], pr[3]);
              dk[2 * i4] = pack_bf16x2(ds[0], ds[1]);
              dk[2 * i4 + 1] = pack_bf16x2(ds[2], ds[3]);
            }
          };
          if (masked)
            body(std::true_type{});
          else
            body(std::false_type{});
          // P^T over its S^T columns; dS^T into the shared buffer (kFuse) and next to P^T, or
          // over the dP^T columns
          tmem_st_x16(tmem + lane_base + cS, pk);
          if constexpr (kFuse) {
            const int nh = 2 * item + h;
            if (nh > 0 && !warp_wait_b(ds_free, (nh - 1) & 1, sAbort, budget)) {
              ok = false;
              break;
            }
            const uint32_t row = smem_u32(sDsT) + (uint32_t)r * 128u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              st_shared_v4(row + 16u * (uint32_t)((4 * wg + j) ^ (r & 7)), dk[4 * j], dk[4 * j + 1],
                           dk[4 * j + 2], dk[4 * j + 3]);
            fence_proxy_async_smem();
            tmem_st_x16(tmem + lane_base + cS + 16, dk);
          } else {
            tmem_st_x16(tmem + lane_base + cS + 64, dk);
          }
          tmem_st_wait();
          tc_fence_before_sync();
          if (!(wg == 0 && h == 0 && item == p.fault_drop_item)) mbar_arrive(&ps_ready[h]);
        }
      }
      if (!ok) break;
      // ---------------------------------------------------------- dV and dK
      // warpgroup wg writes columns [D/2 wg, D/2 (wg + 1)) of dV and dK
      if (n_work > 0) {
        if (!warp_wait_b(acc_done, wk & 1, sAbort, budget)) break;
        tc_fence_after_sync();
        if constexpr (C::kKVinTmem && !kFuse) {
          // the next work's first products may run while this one's dV and dK are written
          // (16 x 16 heads of 64 as above: 56 us, without 60; the same in the dQ kernel, with
          // a barrier more, lost 1 % at heads of 128)
          const PackedWork* y = work_at(w + 1);
          if (y && y->n_work > 0) {
            if (!copy_keys(wk + 1)) break;
            copied = true;
          }
        }
      }
      const int parts = x->parts, head = x->head;
      const long long tok = x->tok_k + r;
#pragma unroll
      for (int which = 0; which < 2; ++which) {  // 0: dV, 1: dK
        const uint32_t acc = tmem + lane_base + (which ? C::kTmAcc1 : C::kTmAcc0) + (D / 2) * wg;
        uint16_t* dst = which ? static_cast<uint16_t*>(p.dk) + tok * p.dk_st + head * p.dk_sh
                              : static_cast<uint16_t*>(p.dv) + tok * p.dv_st + head * p.dv_sh;
        float4* f4 = reinterpret_cast<float4*>(
                         p.sh.key_parts +
                         (((size_t)(x->slot + x->part) * p.H_kv + head) * 2 + which) * kRows * D) +
                     (D / 8) * wg * kRows + r;
#pragma unroll
        for (int ch = 0; ch < D / 64; ++ch) {
          uint32_t v[32];
          if (n_work > 0) {
            tmem_ld_x32(acc + ch * 32, v);
            tmem_ld_wait();
            reg_after_wait(v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;  // no query sees these keys
          }
          if (which == 1 && ch == D / 64 - 1 && n_work > 0) {
            tc_fence_before_sync();
            mbar_arrive(acc_free);
          }
          if (parts > 1) {
#pragma unroll
            for (int qd = 0; qd < 8; ++qd)
              f4[(ch * 8 + qd) * kRows] =
                  make_float4(u2f_b(v[qd * 4 + 0]), u2f_b(v[qd * 4 + 1]),
                              u2f_b(v[qd * 4 + 2]), u2f_b(v[qd * 4 + 3]));
          } else if (r < n_keys) {
            const float mult = which ? p.scale : 1.f;
            uint4* d4 = reinterpret_cast<uint4*>(dst + (D / 2) * wg + ch * 32);
#pragma unroll
            for (int qd = 0; qd < 4; ++qd) {
              uint4 val;
              val.x = pack_bf16x2(u2f_b(v[qd * 8 + 0]) * mult, u2f_b(v[qd * 8 + 1]) * mult);
              val.y = pack_bf16x2(u2f_b(v[qd * 8 + 2]) * mult, u2f_b(v[qd * 8 + 3]) * mult);
              val.z = pack_bf16x2(u2f_b(v[qd * 8 + 4]) * mult, u2f_b(v[qd * 8 + 5]) * mult);
              val.w = pack_bf16x2(u2f_b(v[qd * 8 + 6]) * mult, u2f_b(v[qd * 8 + 7]) * mult);
              d4[qd] = val;
            }
          }
        }
      }
      if (threadIdx.x == 0 && parts > 1) {   // for the end, when the CTA's threads join them
        sParts[*sNumParts] = x->unused[0];
        *sNumParts = *sNumParts + 1;
      }
      if (n_work > 0) ++wk;
      work_done(w);
    }
  } else if (warp == 8) {
    // -------------------------------------------------------- tensor-core issuer
    const bool leader = elect_one();
    const uint64_t dK = kmajor_tile_desc(smem_u32(sK));
    const uint64_t dV = kmajor_tile_desc(smem_u32(sV));
    const uint32_t tS = tmem, tDP = tmem + 64;
    const uint32_t tdV = tmem + C::kTmAcc0, tdK = tmem + C::kTmAcc1;
    int item = 0;
    uint32_t wk = 0;
    bool ok = true;
    for (int w = 0; ok; ++w) {
      const PackedWork* x = work_at(w);
      if (!x) break;
      const int n_work = x->n_work, n_keys = x->n_keys;
      const int first = x->first, tiles = x->tiles, q_len = x->q_len;
      work_done(w);
      if (n_work == 0) continue;
      ok = warp_wait_b(C::kKVinTmem ? kt_ready : kv_full, wk & 1, sAbort, budget);
      if (!ok) break;
      tc_fence_after_sync();
      // What the copies brought from behind the sequence's end, cleared (K for dQ^T = K^T
      // dS^T; a query tile for dV += P^T dO and dK += dS^T Q)
      if (kFuse && n_keys < kRows) clear_rows<D>(sK, n_keys);
      // Q and dO of the work's n-th tile, once they are there
      auto take_tile = [&](int n) {
        const int s = (item + n) % C::kQStages;
        if (!warp_wait_b(&q_full[s], ((item + n) / C::kQStages) & 1, sAbort, budget)) return false;
        tc_fence_after_sync();
        const int rows = (q_len - tile_r0(first, tiles, n)) * group;
        if (rows < group * positions) {
          clear_rows<D>(stage_q(s), rows);
          clear_rows<D>(stage_do(s), rows);
        }
        return true;
      };
      // S^T and dP^T of half h of it, over that half's dQ^T of the tile before once it has been
      // read out
      auto issue_sp = [&](int n, int h) {
        const int i = item + n, s = i % C::kQStages;
        if constexpr (kFuse) {
          if (i > 0 && !warp_wait_b(&dq_free[h], (i - 1) & 1, sAbort, budget)) return false;
          tc_fence_after_sync();
        }
        if (leader) {
          if constexpr (C::kKVinTmem) {
            issue_qk_half_ts<D>(tS + 128 * h, tmem + C::kTmKt, kmajor_tile_desc(smem_u32(stage_q(s))), h);
            issue_qk_half_ts<D>(tDP + 128 * h, tmem + C::kTmVt, kmajor_tile_desc(smem_u32(stage_do(s))), h);
          } else {
            issue_qk_half<D>(tS + 128 * h, dK, kmajor_tile_desc(smem_u32(stage_q(s))), h);
            issue_qk_half<D>(tDP + 128 * h, dV, kmajor_tile_desc(smem_u32(stage_do(s))), h);
          }
          tc_commit(&sp_full[h]);
        }
        return true;
      };
      ok = take_tile(0) && issue_sp(0, 0) && issue_sp(0, 1);
      for (int n = 0; n < n_work && ok; ++n) {
        const int i = item + n, s = i % C::kQStages;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (!warp_wait_b(&ps_ready[h], i & 1, sAbort, budget)) { ok = false; break; }
          // the first products overwrite the dV and dK of the work before
          if (n == 0 && h == 0 && wk > 0 && !warp_wait_b(acc_free, (wk - 1) & 1, sAbort, budget)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          if (leader) {
            if constexpr (kFuse) {
              issue_dqt_half<D>(tDP + 128 * h, mnmajor_tile_desc<D>(smem_u32(sK)),
                                mnmajor_tile_desc<64>(smem_u32(sDsT)));
              tc_commit(&dq_full[h]);
              tc_commit(ds_free);
            }
            issue_pv_half<D>(tdV, tS + 128 * h, mnmajor_tile_desc<D>(smem_u32(stage_do(s))), h,
                             n > 0 || h > 0);
            issue_pv_half<D>(tdK, kFuse ? tS + 128 * h + 16 : tDP + 128 * h,
                             mnmajor_tile_desc<D>(smem_u32(stage_q(s))), h, n > 0 || h > 0);
            if (h == 1) tc_commit(&q_empty[s]);
          }
          if (n + 1 < n_work && ((h == 0 && !take_tile(n + 1)) || !issue_sp(n + 1, h))) {
            ok = false;
            break;
          }
        }
      }
      if (!ok) break;
      if (leader) {
        tc_commit(acc_done);
        tc_commit(kv_free);
      }
      item += n_work;
      ++wk;
    }
    if (leader) {
      tc_commit(drain);
      drain_wait_b(drain, 0, budget);
    }
    __syncwarp();
  } else if (warp == 9) {
    // -------------------------------------------------------- producer
    const bool leader = elect_one();
    const uint64_t pol_kv = l2_policy_evict_first();
    const uint64_t pol_q = l2_policy_evict_last();
    const int entries = p.sh.head->key_blocks;
    int issued = 0;
    uint32_t wk = 0;
    int idx = (int)blockIdx.x;
    bool ok = true;
    for (int w = 0; ok; ++w) {
      PackedWork x = packed_work(p, entries, idx);
      if (w >= 2 && !warp_wait_b(&work_empty[w & 1], ((w >> 1) - 1) & 1, sAbort, budget)) break;
      x.unused[0] = idx;
      if (lane == 0) {
        sWork[w & 1] = x;
        mbar_arrive(&work_full[w & 1]);
      }
      __syncwarp();
      if (!x.valid) break;
      if (x.n_work > 0) {
        // (kept in tensor memory, K and V leave their buffers when they have been copied,
        // unless dQ reads K there)
        uint64_t* const free = C::kKVinTmem && !kFuse ? kt_ready : kv_free;
        if (wk > 0 && !warp_wait_b(free, (wk - 1) & 1, sAbort, budget)) break;
        if (leader) {
          mbar_arrive_expect_tx(kv_full, 2 * C::kTileBytes);
          tma_load_tile<D>(sK, &p.tm_k, kv_full, x.head, x.tok_k, pol_kv);
          tma_load_tile<D>(sV, &p.tm_v, kv_full, x.head, x.tok_k, pol_kv);
        }
        ++wk;
        for (int n = 0; n < x.n_work; ++n) {
          const int s = issued % C::kQStages, round = issued / C::kQStages;
          if (round > 0 && !warp_wait_b(&q_empty[s], (round - 1) & 1, sAbort, budget)) {
            ok = false;
            break;
          }
          if (leader) {
            const int r0 = tile_r0(x.first, x.tiles, n), tok = x.tok_q + r0;
            mbar_arrive_expect_tx(&q_full[s],
                                  (uint32_t)(2 * group * positions * D * 2) + 2 * C::kVecBytes);
            tma_load_tile<D>(stage_q(s), &p.tm_q, &q_full[s], x.head * group, tok, pol_q);
            tma_load_tile<D>(stage_do(s), &p.tm_do, &q_full[s], x.head * group, tok, pol_q);
            const size_t vo =
                (size_t)(x.head * p.vec_stride + (long long)(x.vec0 + r0) * group);
            bulk_load(stage_lse(s), p.nlse2 + vo, C::kVecBytes, &q_full[s]);
            bulk_load(stage_delta(s), p.ndelta + vo, C::kVecBytes, &q_full[s]);
          }
          ++issued;
        }
      }
      // (asked for late, when this work's last tiles are under way: works taken sooner would
      // be bound to a CTA that is long busy)
      if (lane == 0) idx = (int)gridDim.x + atomicAdd(p.sh.next, 1);
      idx = __shfl_sync(kAll, idx, 0);
    }
    if (leader) {
      if (wk > 0) drain_wait_b(kv_full, (wk - 1) & 1, budget);
      const int from = issued > C::kQStages ? issued - C::kQStages : 0;
      for (int t = from; t < issued; ++t)
        drain_wait_b(&q_full[t % C::kQStages], (t / C::kQStages) & 1, budget);
    }
    __syncwarp();
  } else if (kFuse && warp >= 12) {
    // -------------------------------------------------------- dQ read-out
    const bool has_d = (D == 128) || lane < 16;
    const int d = (D == 128) ? (warp & 3) * 32 + lane : (warp & 3) * 16 + (lane & 15);
    float* sStage = reinterpret_cast<float*>(smem + C::kOffDqStage);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    int item = 0, nh = 0;
    bool ok = true;
    for (int w = 0; ok; ++w) {
      const PackedWork* x = work_at(w);
      if constexpr (D == 64) {   // (the four warps meet at barriers below: they leave together)
        if (barrier_or(1, 128, !x)) break;
      } else {
        if (!x) break;
      }
      const int n_work = x->n_work, first = x->first, tiles = x->tiles, q_len = x->q_len;
      // the sequence's first row in the accumulator
      float* rows0 = p.dq_acc + ((long long)x->head * p.sh.T_q + x->tok_q) * group * D;
      work_done(w);
      for (int n = 0; n < n_work && ok; ++n, ++item) {
        const int r0 = tile_r0(first, tiles, n);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if constexpr (D == 64) {
            if (threadIdx.x == 12 * 32) tma_store_wait_read<1>();
          }
          const bool got = warp_wait_b(&dq_full[h], item & 1, sAbort, budget);
          if constexpr (D == 64) {
            if (barrier_or(1, 128, !got)) { ok = false; break; }
          } else {
            if (!got) { ok = false; break; }
          }
          tc_fence_after_sync();
          uint32_t v0[32], v1[32];
          tmem_ld_x32(tmem + lane_base + 128 * h + 64, v0);
          tmem_ld_x32(tmem + lane_base + 128 * h + 96, v1);
          tmem_ld_wait();
          reg_after_wait(v0);
          reg_after_wait(v1);
          tc_fence_before_sync();
          mbar_arrive(&dq_free[h]);
          // rows of the half that exist, and their accumulators
          const int rows = min(q_len - r0, positions) * group - 64 * h;
          float* acc = rows0 + ((long long)r0 * group + 64 * h) * D;
          if constexpr (D == 128) {
            float* dst = acc + d;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < rows) red_add_f32(dst + (size_t)j * D, u2f_b(v0[j]));
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 + j < rows) red_add_f32(dst + (size_t)(32 + j) * D, u2f_b(v1[j]));
          } else {
            float* stg = sStage + (nh & 1) * 64 * D;
            if (has_d) {
#pragma unroll
              for (int j = 0; j < 32; ++j) stg[j * D + d] = u2f_b(v0[j]);
#pragma unroll
              for (int j = 0; j < 32; ++j) stg[(32 + j) * D + d] = u2f_b(v1[j]);
            }
            fence_proxy_async_smem();
            named_barrier_sync(1, 128);
            if (threadIdx.x == 12 * 32) {
              if (rows > 0)
                bulk_reduce_add_f32(acc, smem_u32(stg), (uint32_t)min(rows, 64) * D * 4);
              tma_store_commit();
            }
            ++nh;
          }
        }
      }
    }
    if (D == 64 && threadIdx.x == 12 * 32) tma_store_wait_all();
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 8) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0 && *sAbort) atomicCAS(&g_bwd_status, 0, (int)ATTN_ERR_TIMEOUT);
  if (*sAbort) return;
  // the last of a block's parts adds them up
  for (int i = 0, n = *sNumParts, entries = p.sh.head->key_blocks; i < n; ++i) {
    const PackedWork x = packed_work(p, entries, sParts[i]);
    if (!last_of_parts(p.sh.key_counters + (size_t)x.slot * p.H_kv + x.head, x.parts, sFlag))
      continue;
    const size_t step = (size_t)p.H_kv * 2 * kRows * (D / 4);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const float4* from = reinterpret_cast<const float4*>(
          p.sh.key_parts + (((size_t)x.slot * p.H_kv + x.head) * 2 + which) * kRows * D);
#pragma unroll 1
      for (int j = threadIdx.x; j < ((x.n_keys + 7) & ~7) * (D / 8); j += blockDim.x) {
        int r, c;
        join_item<D>(j, r, c);
        if (r >= x.n_keys) continue;
        float sum[8];
        sum_parts(sum, from + 2 * c * kRows + r, kRows, step, x.parts, [](int) { return 1.f; });
        const long long tok = x.tok_k + r;
        uint16_t* dst = which ? static_cast<uint16_t*>(p.dk) + tok * p.dk_st + x.head * p.dk_sh
                              : static_cast<uint16_t*>(p.dv) + tok * p.dv_st + x.head * p.dv_sh;
        store_bf16x8(dst + c * 8, sum, which ? p.scale : 1.f);
      }
    }
  }
}

// ---------------------------------------------------------------- dQ

template <int D>
__global__ void __launch_bounds__(kThreadsB, 1) attn_bwd_dq_kernel(const __grid_constant__ BwdParams p) {
  using C = BwdCfg<D>;
  extern __shared__ uint8_t smem_raw_b[];
  uint8_t* smem = align_smem_1024(smem_raw_b);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBarQ);
  uint64_t* q_full = bars;
  uint64_t* kv_full = bars + 1;
  uint64_t* kv_empty = kv_full + C::kKVStages;
  uint64_t* sp_full = kv_empty + C::kKVStages;  // [half]: S, dP of the half computed
  uint64_t* ds_ready = sp_full + 2;             // [half]: dS of the half stored
  uint64_t* acc_done = sp_full + 4;
  uint64_t* drain = sp_full + 5;
  uint64_t* qt_ready = sp_full + 6;             // Q and dO copied into tensor memory
  uint32_t* sTmemBase = reinterpret_cast<uint32_t*>(smem + C::kOffMiscQ);
  volatile int* sAbort = reinterpret_cast<volatile int*>(smem + C::kOffMiscQ + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t budget = p.timeout_ns;

  // CTA -> (query block, row group): with the causal mask by cost rank,
  // longest first (with S_q a multiple of 128 a rank is one position block
  // of one head of the group, so the group's heads interleave), in bands
  // (see banded_rank); without it group-major, query blocks last to first
  const int n_qb = (p.R + kRows - 1) / kRows;
  int qb, zkv;
  if (p.causal) {
    int rank;
    banded_rank((int)blockIdx.x, n_qb, p.groups, rank, zkv);
    const int hr = p.R / p.S_q;  // heads per group
    if (p.S_q % kRows == 0) {
      const int nh = p.S_q / kRows;
      qb = (rank % hr) * nh + (nh - 1 - rank / hr);
    } else {
      qb = n_qb - 1 - rank;
    }
  } else {
    zkv = blockIdx.x / n_qb;
    qb = n_qb - 1 - (blockIdx.x - zkv * n_qb);
  }
  const int r0 = qb * kRows;
  int kv_end = p.S_kv;
  if (p.causal) {
    const int last = min(r0 + kRows, p.R) - 1;
    kv_end = min(p.S_kv, (r0 / p.S_q == last / p.S_q) ? last % p.S_q + 1 : p.S_q);
  }
  const int n_kb = (kv_end + kRows - 1) / kRows;   // >= 1: every row sees key 0

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < C::kKVStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sp_full[h], 1);
      mbar_init(&ds_ready[h], 2 * 128);
    }
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    mbar_init(qt_ready, 2 * 128);
    *sAbort = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(sTmemBase, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *sTmemBase;
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sDO = smem + C::kOffDO;
  auto stage_k = [&](int s) { return smem + C::kOffKVRing + s * 2 * C::kTileBytes; };
  auto stage_v = [&](int s) { return stage_k(s) + C::kTileBytes; };

  if (warp < 8) {
    // -------------------------------------------------------- elementwise
    const int w = warp >> 2;                       // key columns 64w .. 64w + 63
    const int r = (warp & 3) * 32 + lane;          // query row within the block
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int rho = r0 + r;
    const bool row_ok = rho < p.R;
    const size_t vo = (size_t)zkv * p.Rp + rho;    // in the padded layout (rho < Rp)
    const uint64_t nlse2x2 = f2_pack(p.nlse2[vo], p.nlse2[vo]);  // -LSE * log2(e), twice
    const uint64_t ndl2 = f2_pack(p.ndelta[vo], p.ndelta[vo]);    // -D_i, twice
    const int pos = rho % p.S_q;
    const int key_limit = p.causal ? min(p.S_kv, pos + 1) : p.S_kv;
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    // Q (warpgroup 0) and dO (warpgroup 1) into tensor memory, the A
    // operands of every S and dP product of this CTA
    bool ok = warp_wait_b(q_full, 0, sAbort, budget);
    if (ok) {
      copy_tile_to_tmem<D>(w == 0 ? sQ : sDO, tmem + lane_base + (w == 0 ? C::kTmQt : C::kTmDOt), r);
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(qt_ready);
    }
    for (int j = 0; j < n_kb && ok; ++j) {
      const int kb0 = j * kRows;
      const bool masked = !row_ok || (kb0 + kRows > key_limit);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (!warp_wait_b(&sp_full[h], j & 1, sAbort, budget)) { ok = false; break; }
        tc_fence_after_sync();
        // half h is keys 64h .. 64h + 63 of the block; this warpgroup's
        // slice is keys 64h + 32w .. 64h + 32w + 31
        const int col0 = 64 * h + 32 * w;
        uint32_t sv[32], dp[32];
        tmem_ld_x32(tmem + lane_base + C::kTmS + col0, sv);
        tmem_ld_x32(tmem + lane_base + C::kTmDP + col0, dp);
        tmem_ld_wait();
        reg_after_wait(sv);
        reg_after_wait(dp);
        uint32_t dk[16];
        // separate masked and unmasked code paths, as in the dK/dV kernel
        auto body = [&](auto masked_tag) {
          constexpr bool kMasked = decltype(masked_tag)::value;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = 2 * i;
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(u2f_b(sv[c]), u2f_b(sv[c + 1])), sl2x2, nlse2x2), x0, x1);
            float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            if constexpr (kMasked) {
              p0 = (row_ok && kb0 + col0 + c < key_limit) ? p0 : 0.f;
              p1 = (row_ok && kb0 + col0 + c + 1 < key_limit) ? p1 : 0.f;
            }
            float d0, d1;
            f2_unpack(f2_mul(f2_pack(p0, p1),
                             f2_add(f2_pack(u2f_b(dp[c]), u2f_b(dp[c + 1])), ndl2)), d0, d1);
            dk[i] = pack_bf16x2(d0, d1);
          }
        };
        if (masked)
          body(std::true_type{});
        else
          body(std::false_type{});
        // dS of the slice: 16 columns from col0 of the S region (this
        // warpgroup's own, already-read columns)
        tmem_st_x16(tmem + lane_base + C::kTmS + col0, dk);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&ds_ready[h]);
      }
    }
    // ---------------------------------------------------------- epilogue
    if (ok && warp_wait_b(acc_done, 0, sAbort, budget)) {
      tc_fence_after_sync();
      uint16_t* dst = static_cast<uint16_t*>(p.dq) + ((size_t)zkv * p.R + rho) * D + (D / 2) * w;
      const uint32_t acc = tmem + lane_base + C::kTmAcc0 + (D / 2) * w;
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch) {
        uint32_t v[32];
        tmem_ld_x32(acc + ch * 32, v);
        tmem_ld_wait();
        reg_after_wait(v);
        if (row_ok) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + ch * 32);
          const float mult = p.scale;
#pragma unroll
          for (int qd = 0; qd < 4; ++qd) {
            uint4 val;
            val.x = pack_bf16x2(u2f_b(v[qd * 8 + 0]) * mult, u2f_b(v[qd * 8 + 1]) * mult);
            val.y = pack_bf16x2(u2f_b(v[qd * 8 + 2]) * mult, u2f_b(v[qd * 8 + 3]) * mult);
            val.z = pack_bf16x2(u2f_b(v[qd * 8 + 4]) * mult, u2f_b(v[qd * 8 + 5]) * mult);
            val.w = pack_bf16x2(u2f_b(v[qd * 8 + 6]) * mult, u2f_b(v[qd * 8 + 7]) * mult);
            d4[qd] = val;
          }
        }
      }
    }
  } else if (warp == 8) {
    // -------------------------------------------------------- tensor-core issuer
    const bool leader = elect_one();
    const uint64_t dQd = kmajor_tile_desc(smem_u32(sQ));
    const uint64_t dOd = kmajor_tile_desc(smem_u32(sDO));
    const uint32_t tS = tmem + C::kTmS, tDP = tmem + C::kTmDP, tdQ = tmem + C::kTmAcc0;
    const uint32_t tQt = tmem + C::kTmQt, tDOt = tmem + C::kTmDOt;
    (void)dQd;
    (void)dOd;
    bool ok = warp_wait_b(qt_ready, 0, sAbort, budget);
    // S and dP of half h of key block j (its K / V stage is loaded), with Q
    // and dO read from tensor memory
    auto issue_sp = [&](int j, int h) {
      const int s = j % C::kKVStages;
      if (leader) {
        issue_qk_half_ts<D>(tS + 64 * h, tQt, kmajor_tile_desc(smem_u32(stage_k(s))), h);
        issue_qk_half_ts<D>(tDP + 64 * h, tDOt, kmajor_tile_desc(smem_u32(stage_v(s))), h);
        tc_commit(&sp_full[h]);
      }
    };
    if (ok && warp_wait_b(&kv_full[0], 0, sAbort, budget)) {
      tc_fence_after_sync();
      issue_sp(0, 0);
      issue_sp(0, 1);
    } else {
      ok = false;
    }
    for (int j = 0; j < n_kb && ok; ++j) {
      const int s = j % C::kKVStages;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (!warp_wait_b(&ds_ready[h], j & 1, sAbort, budget)) { ok = false; break; }
        tc_fence_after_sync();
        if (leader) {
          // dQ += dS K over this half's 64 keys
          issue_pv_half<D>(tdQ, tS + 64 * h, mnmajor_tile_desc<D>(smem_u32(stage_k(s))), h,
                           j > 0 || h > 0);
          if (h == 1) tc_commit(&kv_empty[s]);  // both halves read: the stage is free
        }
        // the next block's half h overwrites the dS these GEMMs read
        if (j + 1 < n_kb) {
          if (h == 0) {
            if (!warp_wait_b(&kv_full[(j + 1) % C::kKVStages], ((j + 1) / C::kKVStages) & 1,
                             sAbort, budget)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
          }
          issue_sp(j + 1, h);
        }
      }
    }
    if (ok && leader) tc_commit(acc_done);
    if (leader) {
      tc_commit(drain);
      drain_wait_b(drain, 0, budget);
    }
    __syncwarp();
  } else if (warp == 9) {
    // -------------------------------------------------------- TMA producer
    const bool leader = elect_one();
    const uint64_t pol_q = l2_policy_evict_first();
    const uint64_t pol_kv = l2_policy_evict_last();
    if (leader) {
      mbar_arrive_expect_tx(q_full, 2 * C::kTileBytes);
      tma_load_tile<D>(sQ, &p.tm_q, q_full, r0, zkv, pol_q);
      tma_load_tile<D>(sDO, &p.tm_do, q_full, r0, zkv, pol_q);
    }
    int issued = 0;
    for (int j = 0; j < n_kb; ++j) {
      const int s = j % C::kKVStages;
      const int round = j / C::kKVStages;
      if (round > 0 && !warp_wait_b(&kv_empty[s], (round - 1) & 1, sAbort, budget)) break;
      if (leader) {
        mbar_arrive_expect_tx(&kv_full[s], 2 * C::kTileBytes);
        tma_load_tile<D>(stage_k(s), &p.tm_k, &kv_full[s], j * kRows, zkv, pol_kv);
        tma_load_tile<D>(stage_v(s), &p.tm_v, &kv_full[s], j * kRows, zkv, pol_kv);
      }
      ++issued;
    }
    if (leader) {
      drain_wait_b(q_full, 0, budget);
      const int first = issued > C::kKVStages ? issued - C::kKVStages : 0;
      for (int t = first; t < issued; ++t)
        drain_wait_b(&kv_full[t % C::kKVStages], (t / C::kKVStages) & 1, budget);
    }
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 8) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0 && *sAbort) atomicCAS(&g_bwd_status, 0, (int)ATTN_ERR_TIMEOUT);
}

// ---------------------------------------------------------------- dQ, packed

// One work item of the kernel below: 128 rows (half a tile of the list) of a K/V head, or a
// part of their keys.
struct PackedDqWork {
  int valid;
  int rows, tok_q, vec0;                 // rows that exist (0: an empty half), their first token
  int tok_k, k_len, n_keys, diag;        // as in PackedTile, of the half
  int jb, n_blocks;                      // its key blocks
  int part, parts, slot;                 // slot: of the tile's first part and the head
  int head, half;
  int idx;
};
static_assert(sizeof(PackedDqWork) == 64 && sizeof(PackedWork) == 64, "slots of shared memory");

__device__ __forceinline__ PackedDqWork packed_dq_work(const PackedBwdParams& p, int entries,
                                                       int idx) {
  PackedDqWork x;
  x.idx = idx;
  x.half = idx & 1;
  x.valid = (long long)(idx >> 1) < (long long)entries * p.H_kv;
  if (!x.valid) return x;
  int entry;
  banded_rank<kPackedBand>(idx >> 1, entries, p.H_kv, entry, x.head);
  const int positions = p.sh.positions, at = x.half * positions;
  const int4* src = reinterpret_cast<const int4*>(p.sh.tiles + entry);
  const int4 a = src[0], b = src[1], c = src[2];   // in PackedTile's order
  const int tokens = max(min(a.y - at, positions), 0);
  x.rows = tokens * p.sh.group;
  x.tok_q = a.x + at;
  x.tok_k = a.z;
  x.k_len = a.w;
  x.diag = b.y + at;
  x.vec0 = b.z + at;
  x.jb = b.w;
  x.parts = c.y;
  x.part = c.z;
  x.slot = c.w * p.H_kv + x.head;
  // (a half may see fewer keys than the tile)
  x.n_keys = p.causal ? min(max(x.diag + tokens - 1, 0), x.k_len) : x.k_len;
  x.n_blocks = max(min((x.n_keys + kRows - 1) / kRows, x.jb + c.x) - x.jb, 0);
  return x;
}

// attn_bwd_dq_kernel over packed sequences, persistent as packed_bwd_dkdv_kernel is and with
// the same counter and slots: while the dQ of one work is written, the producer has the
// next one's Q and dO in shared memory (free as soon as they have been copied into tensor
// memory) and its first keys in the ring.  Beside attn_bwd_dq_kernel's barriers
//   qt_ready   also tells the issuer that the dQ before has been read out
//   work_full, work_empty [slot]
// The order of a row's sums does not depend on which thread block does a work.  In bands of
// four tiles the costliest run first where there are few, and a head's keys are still
// shared in L2 (bands of 16, 4 and 1: the cross attention below 109.5, 99.6, 99.2 us; one
// sequence of 16384 tokens 5295, 5176, 5226).
//
// Bound by the chain of hand-offs, as packed_bwd_dkdv_kernel.  Deterministic gradients of
// 16 x 1024 tokens, 32 heads over 8 of 128, causal: 546 us in all, 613 with a thread block
// to each half of a tile; 64 x 256 tokens 300 and 367; 16 x 16 heads of 64, queries of
// 20 to 1000 tokens over keys of 64 to 2304, 100 and 121 (96 now).
template <int D>
__global__ void __launch_bounds__(kThreadsB, 1)
    packed_bwd_dq_kernel(const __grid_constant__ PackedBwdParams p) {
  using C = BwdCfg<D>;
  extern __shared__ uint8_t smem_raw_b[];
  uint8_t* smem = align_smem_1024(smem_raw_b);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBarQ);
  uint64_t* q_full = bars;
  uint64_t* kv_full = bars + 1;
  uint64_t* kv_empty = kv_full + C::kKVStages;
  uint64_t* sp_full = kv_empty + C::kKVStages;
  uint64_t* ds_ready = sp_full + 2;
  uint64_t* acc_done = sp_full + 4;
  uint64_t* drain = sp_full + 5;
  uint64_t* qt_ready = sp_full + 6;
  uint64_t* work_full = sp_full + 7;
  uint64_t* work_empty = sp_full + 9;
  uint32_t* sTmemBase = reinterpret_cast<uint32_t*>(smem + C::kOffMiscQ);
  volatile int* sAbort = reinterpret_cast<volatile int*>(smem + C::kOffMiscQ + 4);
  volatile int* sFlag = reinterpret_cast<volatile int*>(smem + C::kOffMiscQ + 8);
  volatile int* sNumParts = reinterpret_cast<volatile int*>(smem + C::kOffMiscQ + 12);
  PackedDqWork* sWork = reinterpret_cast<PackedDqWork*>(smem + C::kOffWorkQ);
  int* sParts = reinterpret_cast<int*>(smem + C::kOffWorkQ + 2 * sizeof(PackedDqWork));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t budget = p.timeout_ns;
  const int group = p.sh.group, positions = p.sh.positions;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < C::kKVStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sp_full[h], 1);
      mbar_init(&ds_ready[h], 2 * 128);
      mbar_init(&work_full[h], 1);
      mbar_init(&work_empty[h], 9);   // warps 0-8
    }
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    mbar_init(qt_ready, 2 * 128);
    *sAbort = 0;
    *sNumParts = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(sTmemBase, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *sTmemBase;
  wait_for_earlier();
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sDO = smem + C::kOffDO;
  auto stage_k = [&](int s) { return smem + C::kOffKVRing + s * 2 * C::kTileBytes; };
  auto stage_v = [&](int s) { return stage_k(s) + C::kTileBytes; };
  // the w-th work of this CTA, once it is known; nullptr behind the last (or when a wait
  // ran out)
  auto work_at = [&](int w) -> const PackedDqWork* {
    if (!warp_wait_b(&work_full[w & 1], (w >> 1) & 1, sAbort, budget)) return nullptr;
    const PackedDqWork* x = sWork + (w & 1);
    return x->valid ? x : nullptr;
  };
  auto work_done = [&](int w) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&work_empty[w & 1]);
  };
  // the float4s of a part's dQ
  auto part_of = [&](const PackedDqWork& x, int part) {
    return reinterpret_cast<float4*>(
        p.sh.tile_parts + ((x.slot + (size_t)part * p.H_kv) * 256 + x.half * kRows) * D);
  };

  if (warp < 8) {
    // -------------------------------------------------------- elementwise
    const int wg = warp >> 2;                      // key columns 32 wg .. 32 wg + 31 of a half
    const int r = (warp & 3) * 32 + lane;          // query row within the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int at = (r * p.sh.inv_group) >> 16;     // its query token
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    int item = 0;                                  // key blocks so far
    uint32_t wk = 0;                               // works with any so far
    bool ok = true;
    for (int w = 0; ok; ++w) {
      const PackedDqWork* x = work_at(w);
      if (!x) break;
      const int n_blocks = x->n_blocks;
      const bool row_ok = r < x->rows;
      if (n_blocks > 0) {
        // (the vectors go on behind the last tile)
        const size_t vo = (size_t)(x->head * p.vec_stride + (long long)x->vec0 * group + r);
        const float nlse2 = p.nlse2[vo], ndl = p.ndelta[vo];   // -LSE * log2(e), -D_i
        const uint64_t nlse2x2 = f2_pack(nlse2, nlse2), ndl2 = f2_pack(ndl, ndl);
        const int key_limit =
            !row_ok ? 0 : p.causal ? min(x->n_keys, x->diag + at) : x->n_keys;
        // Q (warpgroup 0) and dO (warpgroup 1) into tensor memory; the products of the work
        // before, which read them there, are done (acc_done below)
        ok = warp_wait_b(q_full, wk & 1, sAbort, budget);
        if (!ok) break;
        copy_tile_to_tmem<D>(wg == 0 ? sQ : sDO,
                             tmem + lane_base + (wg == 0 ? C::kTmQt : C::kTmDOt), r);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(qt_ready);
        const int key0 = x->jb * kRows;
        for (int j = 0; j < n_blocks && ok; ++j, ++item) {
          const int kb0 = key0 + j * kRows;
          const bool masked = kb0 + kRows > key_limit;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (!warp_wait_b(&sp_full[h], item & 1, sAbort, budget)) { ok = false; break; }
            tc_fence_after_sync();
            const int col0 = 64 * h + 32 * wg;
            uint32_t sv[32], dp[32];
            tmem_ld_x32(tmem + lane_base + C::kTmS + col0, sv);
            tmem_ld_x32(tmem + lane_base + C::kTmDP + col0, dp);
            tmem_ld_wait();
            reg_after_wait(sv);
            reg_after_wait(dp);
            uint32_t dk[16];
            auto body = [&](auto masked_tag) {
              constexpr bool kMasked = decltype(masked_tag)::value;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int c = 2 * i;
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(u2f_b(sv[c]), u2f_b(sv[c + 1])), sl2x2, nlse2x2), x0, x1);
                float d0, d1;
                f2_unpack(f2_mul(f2_pack(ex2_approx(x0), ex2_approx(x1)),
                                 f2_add(f2_pack(u2f_b(dp[c]), u2f_b(dp[c + 1])), ndl2)), d0, d1);
                if constexpr (kMasked) {
                  // (what a masked S or dP holds may be another sequence's infinity)
                  d0 = kb0 + col0 + c < key_limit ? d0 : 0.f;
                  d1 = kb0 + col0 + c + 1 < key_limit ? d1 : 0.f;
                }
                dk[i] = pack_bf16x2(d0, d1);
              }
            };
            if (masked)
              body(std::true_type{});
            else
              body(std::false_type{});
            // dS over the slice's own columns of S, which have been read
            tmem_st_x16(tmem + lane_base + C::kTmS + col0, dk);
            tmem_st_wait();
            tc_fence_before_sync();
            if (!(wg == 0 && h == 0 && item == p.fault_drop_item)) mbar_arrive(&ds_ready[h]);
          }
        }
        if (!ok) break;
        if (!warp_wait_b(acc_done, wk & 1, sAbort, budget)) break;
        tc_fence_after_sync();
        ++wk;
      }
      // ---------------------------------------------------------- dQ
      // warpgroup wg writes columns [D/2 wg, D/2 (wg + 1))
      const uint32_t acc = tmem + lane_base + C::kTmAcc0 + (D / 2) * wg;
      const int parts = x->parts;
      float4* f4 = part_of(*x, x->part) + (D / 8) * wg * kRows + r;
      uint16_t* dst = static_cast<uint16_t*>(p.dq) + (long long)(x->tok_q + at) * p.dq_st +
                      (x->head * group + r - at * group) * p.dq_sh + (D / 2) * wg;
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch) {
        uint32_t v[32];
        if (n_blocks > 0) {
          tmem_ld_x32(acc + ch * 32, v);
          tmem_ld_wait();
          reg_after_wait(v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;   // no row sees a key of these
        }
        if (parts > 1) {
#pragma unroll
          for (int qd = 0; qd < 8; ++qd)
            f4[(ch * 8 + qd) * kRows] = make_float4(u2f_b(v[qd * 4 + 0]), u2f_b(v[qd * 4 + 1]),
                                                    u2f_b(v[qd * 4 + 2]), u2f_b(v[qd * 4 + 3]));
        } else if (row_ok) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + ch * 32);
          const float mult = p.scale;
#pragma unroll
          for (int qd = 0; qd < 4; ++qd) {
            uint4 val;
            val.x = pack_bf16x2(u2f_b(v[qd * 8 + 0]) * mult, u2f_b(v[qd * 8 + 1]) * mult);
            val.y = pack_bf16x2(u2f_b(v[qd * 8 + 2]) * mult, u2f_b(v[qd * 8 + 3]) * mult);
            val.z = pack_bf16x2(u2f_b(v[qd * 8 + 4]) * mult, u2f_b(v[qd * 8 + 5]) * mult);
            val.w = pack_bf16x2(u2f_b(v[qd * 8 + 6]) * mult, u2f_b(v[qd * 8 + 7]) * mult);
            d4[qd] = val;
          }
        }
      }
      tc_fence_before_sync();   // (dQ is read out before qt_ready of the next work)
      if (threadIdx.x == 0 && parts > 1) {   // for the end, when the CTA's threads join them
        sParts[*sNumParts] = x->idx;
        *sNumParts = *sNumParts + 1;
      }
      work_done(w);
    }
  } else if (warp == 8) {
    // -------------------------------------------------------- tensor-core issuer
    const bool leader = elect_one();
    const uint32_t tS = tmem + C::kTmS, tDP = tmem + C::kTmDP, tdQ = tmem + C::kTmAcc0;
    const uint32_t tQt = tmem + C::kTmQt, tDOt = tmem + C::kTmDOt;
    int item = 0;
    uint32_t wk = 0;
    bool ok = true;
    for (int w = 0; ok; ++w) {
      const PackedDqWork* x = work_at(w);
      if (!x) break;
      const int n_blocks = x->n_blocks, left = x->k_len - x->jb * kRows;
      work_done(w);
      if (n_blocks == 0) continue;
      ok = warp_wait_b(qt_ready, wk & 1, sAbort, budget);
      if (!ok) break;
      tc_fence_after_sync();
      // K and V of the work's j-th block, once they are there; rows of K behind the sequence's
      // end cleared, for dQ += dS K
      auto take_keys = [&](int j) {
        const int s = (item + j) % C::kKVStages;
        if (!warp_wait_b(&kv_full[s], ((item + j) / C::kKVStages) & 1, sAbort, budget)) return false;
        tc_fence_after_sync();
        if (left - j * kRows < kRows) clear_rows<D>(stage_k(s), left - j * kRows);
        return true;
      };
      // S and dP of half h of it, with Q and dO read from tensor memory
      auto issue_sp = [&](int j, int h) {
        const int s = (item + j) % C::kKVStages;
        if (leader) {
          issue_qk_half_ts<D>(tS + 64 * h, tQt, kmajor_tile_desc(smem_u32(stage_k(s))), h);
          issue_qk_half_ts<D>(tDP + 64 * h, tDOt, kmajor_tile_desc(smem_u32(stage_v(s))), h);
          tc_commit(&sp_full[h]);
        }
      };
      ok = take_keys(0);
      if (!ok) break;
      issue_sp(0, 0);
      issue_sp(0, 1);
      for (int j = 0; j < n_blocks && ok; ++j) {
        const int i = item + j, s = i % C::kKVStages;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (!warp_wait_b(&ds_ready[h], i & 1, sAbort, budget)) { ok = false; break; }
          tc_fence_after_sync();
          if (leader) {
            issue_pv_half<D>(tdQ, tS + 64 * h, mnmajor_tile_desc<D>(smem_u32(stage_k(s))), h,
                             j > 0 || h > 0);
            if (h == 1) tc_commit(&kv_empty[s]);
          }
          if (j + 1 < n_blocks) {
            if (h == 0 && !take_keys(j + 1)) { ok = false; break; }
            issue_sp(j + 1, h);
          }
        }
      }
      if (!ok) break;
      if (leader) tc_commit(acc_done);
      item += n_blocks;
      ++wk;
    }
    if (leader) {
      tc_commit(drain);
      drain_wait_b(drain, 0, budget);
    }
    __syncwarp();
  } else if (warp == 9) {
    // -------------------------------------------------------- producer
    const bool leader = elect_one();
    const uint64_t pol_q = l2_policy_evict_first();
    const uint64_t pol_kv = l2_policy_evict_last();
    const int entries = p.sh.head->tiles;
    int issued = 0;
    uint32_t wk = 0;
    int idx = (int)blockIdx.x;
    auto claim = [&]() {
      if (lane == 0) idx = (int)gridDim.x + atomicAdd(p.sh.next + 1, 1);
      idx = __shfl_sync(kAll, idx, 0);
    };
    bool ok = true;
    for (int w = 0; ok; ++w) {
      PackedDqWork x = packed_dq_work(p, entries, idx);
      while (x.valid && x.rows == 0) {   // an empty half
        claim();
        x = packed_dq_work(p, entries, idx);
      }
      if (w >= 2 && !warp_wait_b(&work_empty[w & 1], ((w >> 1) - 1) & 1, sAbort, budget)) break;
      if (lane == 0) {
        sWork[w & 1] = x;
        mbar_arrive(&work_full[w & 1]);
      }
      __syncwarp();
      if (!x.valid) break;
      if (x.n_blocks > 0) {
        if (wk > 0 && !warp_wait_b(qt_ready, (wk - 1) & 1, sAbort, budget)) break;
        if (leader) {
          mbar_arrive_expect_tx(q_full, (uint32_t)(2 * group * positions * D * 2));
          tma_load_tile<D>(sQ, &p.tm_q, q_full, x.head * group, x.tok_q, pol_q);
          tma_load_tile<D>(sDO, &p.tm_do, q_full, x.head * group, x.tok_q, pol_q);
        }
        ++wk;
        for (int j = 0; j < x.n_blocks; ++j) {
          const int s = issued % C::kKVStages, round = issued / C::kKVStages;
          if (round > 0 && !warp_wait_b(&kv_empty[s], (round - 1) & 1, sAbort, budget)) {
            ok = false;
            break;
          }
          if (leader) {
            const int tok = x.tok_k + (x.jb + j) * kRows;
            mbar_arrive_expect_tx(&kv_full[s], 2 * C::kTileBytes);
            tma_load_tile<D>(stage_k(s), &p.tm_k, &kv_full[s], x.head, tok, pol_kv);
            tma_load_tile<D>(stage_v(s), &p.tm_v, &kv_full[s], x.head, tok, pol_kv);
          }
          ++issued;
        }
      }
      claim();   // (late, as in packed_bwd_dkdv_kernel)
    }
    if (leader) {
      if (wk > 0) drain_wait_b(q_full, (wk - 1) & 1, budget);
      const int from = issued > C::kKVStages ? issued - C::kKVStages : 0;
      for (int t = from; t < issued; ++t)
        drain_wait_b(&kv_full[t % C::kKVStages], (t / C::kKVStages) & 1, budget);
    }
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 8) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0 && *sAbort) atomicCAS(&g_bwd_status, 0, (int)ATTN_ERR_TIMEOUT);
  if (*sAbort) return;
  // the last of a tile's parts adds them up
  for (int i = 0, n = *sNumParts, entries = p.sh.head->tiles; i < n; ++i) {
    const PackedDqWork x = packed_dq_work(p, entries, sParts[i]);
    if (!last_of_parts(p.sh.tile_counters + (size_t)x.slot * 2 + x.half, x.parts, sFlag)) continue;
    const float4* from = part_of(x, 0);
#pragma unroll 1
    for (int j = threadIdx.x; j < ((x.rows + 7) & ~7) * (D / 8); j += kThreadsB) {
      int r, c;
      join_item<D>(j, r, c);
      if (r >= x.rows) continue;
      const int at = (r * p.sh.inv_group) >> 16;
      float sum[8];
      sum_parts(sum, from + 2 * c * kRows + r, kRows, (size_t)p.H_kv * 256 * (D / 4), x.parts,
                [](int) { return 1.f; });
      store_bf16x8(static_cast<uint16_t*>(p.dq) + (long long)(x.tok_q + at) * p.dq_st +
                       (x.head * group + r - at * group) * p.dq_sh + c * 8,
                   sum, p.scale);
    }
  }
}

namespace {

std::mutex g_bwd_mu;
bool g_bwd_attr[2][64] = {};  // [D == 128][device]

template <int D, bool kFuse>
cudaError_t set_dkdv_attr() {
  return cudaFuncSetAttribute(attn_bwd_dkdv_kernel<D, kFuse>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, BwdCfg<D>::kSmemKV);
}

template <int D>
cudaError_t launch_bwd_d(const BwdParams& p, const void* o, const void* dout, const float* lse,
                         cudaStream_t stream) {
  using C = BwdCfg<D>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_bwd_mu);
    if (!g_bwd_attr[D == 128][dev]) {
      err = set_dkdv_attr<D, false>();
      if (err != cudaSuccess) return err;
      err = set_dkdv_attr<D, true>();
      if (err != cudaSuccess) return err;
      err = cudaFuncSetAttribute(attn_bwd_dq_kernel<D>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemQ);
      if (err != cudaSuccess) return err;
      g_bwd_attr[D == 128][dev] = true;
    }
  }
  const long long prep_rows = (long long)p.groups * p.Rp;
  const long long prep_rows_per_block = 8 * kPrepRowsPerWarp;
  attn_bwd_prep_kernel<D><<<(unsigned)((prep_rows + prep_rows_per_block - 1) / prep_rows_per_block),
                            256, 0, stream>>>(
      p, static_cast<const uint16_t*>(o), static_cast<const uint16_t*>(dout), lse);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const unsigned grid_kv = (unsigned)((p.S_kv + kRows - 1) / kRows) * (unsigned)p.groups;
  if (p.dq_acc != nullptr) {
    attn_bwd_dkdv_kernel<D, true><<<grid_kv, kThreadsFused, C::kSmemKV, stream>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const long long pieces = (long long)p.groups * p.R * (D / 8);
    attn_bwd_dq_convert_kernel<D><<<(unsigned)((pieces + 255) / 256), 256, 0, stream>>>(p);
    return cudaGetLastError();
  }
  attn_bwd_dkdv_kernel<D, false><<<grid_kv, kThreadsB, C::kSmemKV, stream>>>(p);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const unsigned grid_q = (unsigned)((p.R + kRows - 1) / kRows) * (unsigned)p.groups;
  attn_bwd_dq_kernel<D><<<grid_q, kThreadsB, C::kSmemQ, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_packed_bwd_d(const PackedBwdParams& p, const PackedPlan& plan, const void* o,
                                const void* dout, const float* lse, int tile_room, int key_room,
                                cudaStream_t stream) {
  using C = BwdCfg<D>;
  static bool attr_set[64] = {};   // (of this head dimension, by device)
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_bwd_mu);
    if (!attr_set[dev]) {
      constexpr auto kAttr = cudaFuncAttributeMaxDynamicSharedMemorySize;
      if ((err = cudaFuncSetAttribute(packed_bwd_dkdv_kernel<D, false>, kAttr, C::kSmemKV)) !=
              cudaSuccess ||
          (err = cudaFuncSetAttribute(packed_bwd_dkdv_kernel<D, true>, kAttr, C::kSmemKV)) !=
              cudaSuccess ||
          (err = cudaFuncSetAttribute(packed_bwd_dq_kernel<D>, kAttr, C::kSmemQ)) != cudaSuccess)
        return err;
      attr_set[dev] = true;
    }
  }
  const long long rows = (long long)p.sh.T_q * p.H_q, rows_per_block = 8 * kPrepRowsPerWarp;
  const dim3 prep((unsigned)((rows + rows_per_block - 1) / rows_per_block));
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = prep;
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (!plan.early && (err = launch_packed_plan(plan, stream)) != cudaSuccess) return err;
  err = cudaLaunchKernelEx(&cfg, packed_bwd_prep_kernel<D>, p, static_cast<const uint16_t*>(o),
                           static_cast<const uint16_t*>(dout), lse);
  if (err != cudaSuccess) return err;
  if (plan.early && (err = launch_packed_plan(plan, stream)) != cudaSuccess) return err;
  // persistent: one CTA per SM
  int sms = 0;
  if ((err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return err;
  const long long works = (long long)key_room * p.H_kv;
  const dim3 grid_kv((unsigned)(works < sms ? works : sms));
  if (p.dq_acc != nullptr) {
    err = launch_ahead(packed_bwd_dkdv_kernel<D, true>, grid_kv, kThreadsFused, C::kSmemKV,
                       stream, p);
    if (err != cudaSuccess) return err;
    const long long per_head = (long long)p.sh.T_q * p.sh.group * (D / 8);
    return launch_ahead(packed_bwd_dq_convert_kernel<D>,
                        dim3((unsigned)((per_head + 255) / 256), (unsigned)p.H_kv), 256, 0, stream, p);
  }
  err = launch_ahead(packed_bwd_dkdv_kernel<D, false>, grid_kv, kThreadsB, C::kSmemKV, stream, p);
  if (err != cudaSuccess) return err;
  const long long halves = (long long)tile_room * p.H_kv * 2;
  return launch_ahead(packed_bwd_dq_kernel<D>, dim3((unsigned)(halves < sms ? halves : sms)),
                      kThreadsB, C::kSmemQ, stream, p);
}

}  // namespace

cudaError_t launch_attn_bwd_packed(const PackedBwdParams& p, const PackedPlan& plan, int D,
                                   const void* o, const void* dout, const float* lse,
                                   int tile_room, int key_room, cudaStream_t stream) {
  if (D == 128) return launch_packed_bwd_d<128>(p, plan, o, dout, lse, tile_room, key_room, stream);
  if (D == 64) return launch_packed_bwd_d<64>(p, plan, o, dout, lse, tile_room, key_room, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_attn_bwd(const BwdParams& p, int D, const void* o, const void* dout,
                            const float* lse, cudaStream_t stream) {
  if (D == 128) return launch_bwd_d<128>(p, o, dout, lse, stream);
  if (D == 64) return launch_bwd_d<64>(p, o, dout, lse, stream);
  return cudaErrorInvalidValue;
}

cudaError_t read_bwd_status(int* status, bool reset) {
  cudaError_t err = cudaMemcpyFromSymbol(status, g_bwd_status, sizeof(int));
  if (err != cudaSuccess) return err;
  if (reset) {
    const int zero = 0;
    err = cudaMemcpyToSymbol(g_bwd_status, &zero, sizeof(int));
  }
  return err;
}

}  // namespace attnpipe
