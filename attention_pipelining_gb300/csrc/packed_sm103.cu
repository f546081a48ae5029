// packed_sm103.cu -- packed sequences: the plan of their attention's work, and
// the rotation of queries and keys by positions with several axes
// (include/attn_packed.h).
#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "rotate.cuh"

namespace attnpipe {

__device__ int g_packed_status = 0;

namespace {

// ---------------------------------------------------------------- plan

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;   // of costs

// Sum (or maximum) over the warp's lanes up to this one.
template <typename Op>
__device__ __forceinline__ int warp_scan(int x, Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x = op(x, y);
  }
  return x;
}

// The scan over the block's threads before this one (`none` for the first); `warps`: 32
// ints of shared memory.
template <typename Op>
__device__ __forceinline__ int block_scan_before(int x, int none, int* warps, Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int upto = warp_scan(x, op);
  __syncthreads();   // (warps may still be read from the scan before)
  if (lane == 31) warps[warp] = upto;
  __syncthreads();
  if (warp == 0) warps[lane] = warp_scan(warps[lane], op);
  __syncthreads();
  int before = __shfl_up_sync(0xffffffffu, upto, 1);
  if (lane == 0) before = none;
  return warp > 0 ? op(warps[warp - 1], before) : before;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// cu in order, within [0, T]: each entry the largest up to there.  True if it was not.
__device__ bool put_in_order(const int* cu, int n, int T, int* out, int* warps) {
  const auto larger = [](int a, int b) { return max(a, b); };
  const int per = ceil_div(n, kPlanThreads);
  const int first = min((int)threadIdx.x * per, n), end = min(first + per, n);
  int most = 0;
  for (int i = first; i < end; ++i) most = max(most, min(cu[i], T));
  int run = block_scan_before(most, 0, warps, larger);
  bool bad = false;
  for (int i = first; i < end; ++i) {
    const int x = cu[i];
    run = max(run, min(x, T));
    bad |= x != run;
    out[i] = run;
  }
  return bad;
}

// Into how many parts an entry of n blocks is cut (see kPackedCtas).
__device__ __forceinline__ int parts_of(int n, int cap) {
  return 2 * n >= 3 * cap ? (n + cap / 2) / cap : 1;
}

// One thread block lists the tiles and the key blocks of all sequences, by a
// counting sort over their costs in blocks (of 128 keys, or of query tiles), so that
// the costliest run first and the last to end are short.  The order among equal costs
// and the parts' slots differ from run to run; no result depends on them.
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PackedPlan p) {
  __shared__ int at[2][kBuckets];   // entries of a cost, then where the next of them goes
  __shared__ int warps[32], most[2], slots[2];
  __shared__ unsigned long long total[2];   // blocks of all entries
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  at[0][threadIdx.x] = at[1][threadIdx.x] = 0;
  if (threadIdx.x < 2) most[threadIdx.x] = slots[threadIdx.x] = 0, total[threadIdx.x] = 0;
  allow_later();
  wait_for_earlier();
  bool bad = put_in_order(p.cu_q, p.B + 1, p.T_q, p.seq_q, warps);
  if (p.seq_k != p.seq_q) bad |= put_in_order(p.cu_k, p.B + 1, p.T_k, p.seq_k, warps);
  if (bad) g_packed_status = ATTN_ERR_BAD_INDEX;
  __syncthreads();
  const int P = p.positions;
  for (int b = threadIdx.x; b < p.B; b += kPlanThreads) {
    const int n = p.seq_q[b + 1] - p.seq_q[b], m = p.seq_k[b + 1] - p.seq_k[b];
    if (n > 0) atomicMax(&most[0], ceil_div(m, 128));
    if (m > 0) atomicMax(&most[1], ceil_div(n, P));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    for (int c = threadIdx.x; c < p.n_counters; c += kPlanThreads)
      if (p.counters[i] != nullptr) p.counters[i][c] = 0;
  // every tile (list 0) and key block (list 1), whole, each with its cost
  const auto each = [&](auto&& put) {
    for (int b = warp; b < p.B; b += kPlanThreads / 32) {
      const int q0 = p.seq_q[b], n = p.seq_q[b + 1] - q0;
      const int k0 = p.seq_k[b], m = p.seq_k[b + 1] - k0;
      const int vec0 = packed_vec0(q0, b);
      for (int t = lane; p.tiles != nullptr && t < ceil_div(n, 2 * P); t += 32) {
        PackedTile x;
        const int pos = t * 2 * P;
        x.tok0 = q0 + pos;
        x.rows = min(n - pos, 2 * P);
        x.k0 = k0;
        x.k_len = m;
        x.diag = m - n + pos + 1;
        x.n_keys = p.causal ? min(max(x.diag + x.rows - 1, 0), m) : m;
        x.vec0 = vec0 + pos;
        put(0, ceil_div(x.n_keys, 128), &x, (PackedKeys*)nullptr);
      }
      if (p.keys == nullptr) continue;
      const int tiles = ceil_div(n, P);
      for (int t = lane; t < ceil_div(m, 128); t += 32) {
        PackedKeys x;
        x.k0 = k0 + t * 128;
        x.keys = min(m - t * 128, 128);
        x.q0 = q0;
        x.q_len = n;
        x.vec0 = vec0;
        x.shift = t * 128 - (m - n);
        // (without a mask each block begins elsewhere, so that those that run at once
        // add to different rows of dQ)
        x.first = p.causal ? min(max(x.shift, 0) / P, tiles) : tiles > 0 ? t % tiles : 0;
        x.n_work = p.causal ? tiles - x.first : tiles;
        x.tiles = tiles;
        put(1, x.n_work, (PackedTile*)nullptr, &x);
      }
    }
  };
  int shift[2], cap[2];
  const bool may_cut = 2 * max(most[0], most[1]) >= 3 * kPackedLeastPart;
  if (may_cut) {
    unsigned long long mine[2] = {0, 0};
    each([&](int list, int cost, PackedTile*, PackedKeys*) { mine[list] += cost; });
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mine[i] += __shfl_xor_sync(0xffffffffu, mine[i], off);
      if (lane == 0 && mine[i] > 0) atomicAdd(&total[i], mine[i]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned long long share = (total[i] * p.H_kv + kPackedCtas - 1) / kPackedCtas;
    cap[i] = may_cut ? (int)min(max(share, (unsigned long long)kPackedLeastPart), 1ull << 29) : 1 << 29;
    shift[i] = 0;
    while ((most[i] >> shift[i]) >= kBuckets) ++shift[i];
  }
  const auto bucket = [&](int list, int cost) {
    return &at[list][kBuckets - 1 - min(cost >> shift[list], kBuckets - 1)];
  };
  // an entry of n blocks has `parts` parts of `size` blocks, but for the last
  const auto cut = [&](int list, int n, int& parts, int& size) {
    parts = parts_of(n, cap[list]);
    size = ceil_div(n, parts);
    parts = n > 0 ? ceil_div(n, size) : 1;
  };
  each([&](int list, int cost, PackedTile*, PackedKeys*) {
    int parts, size;
    cut(list, cost, parts, size);
    if (parts > 1) atomicAdd(bucket(list, size), parts - 1);
    atomicAdd(bucket(list, cost - (parts - 1) * size), 1);
  });
  __syncthreads();
  const auto sum = [](int a, int b) { return a + b; };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int mine = at[i][threadIdx.x];
    const int before = block_scan_before(mine, 0, warps, sum);
    at[i][threadIdx.x] = before;
    if (threadIdx.x == kBuckets - 1) {
      if (i == 0) p.head->tiles = before + mine;
      if (i == 1) p.head->key_blocks = before + mine;
    }
  }
  if (threadIdx.x == 0) {
    p.head->q_first = p.seq_q[0];
    p.head->q_end = p.seq_q[p.B];
    p.head->cut = 2 * most[0] >= 3 * cap[0];
  }
  __syncthreads();
  each([&](int list, int cost, PackedTile* tile, PackedKeys* keys) {
    int parts, size;
    cut(list, cost, parts, size);
    const int slot = parts > 1 ? atomicAdd(&slots[list], parts) : 0;
    const int first = list == 1 ? keys->first : 0;
    for (int part = 0; part < parts; ++part) {
      const int n = part + 1 < parts ? size : cost - part * size;
      const int i = atomicAdd(bucket(list, n), 1);
      if (list == 0) {
        tile->jb = part * size, tile->n_blocks = n;
        tile->parts = parts, tile->part = part, tile->slot = slot;
        p.tiles[i] = *tile;
      } else {
        const int t = first + part * size;
        keys->first = t < keys->tiles ? t : t - keys->tiles, keys->n_work = n;
        keys->parts = parts, keys->part = part, keys->slot = slot;
        p.keys[i] = *keys;
      }
    }
  });
}
static_assert(kBuckets == kPlanThreads, "one thread to a bucket");

// ---------------------------------------------------------------- rotation

constexpr int kRopeThreads = 128;
constexpr int kRopeAhead = 4;        // rows of a thread under way
constexpr int kRopeResident = 6;     // thread blocks on an SM
constexpr int kRopeWave = kRopeResident * 152;

// A token's vector of one head is a row that D / 16 neighbouring lanes hold, 16
// elements each: eight first and eight second elements of their pairs, or (adjacent
// pairs, or not rotated) eight of either half of the row.  A thread block takes kSlots consecutive
// tokens and goes with all of them through p.rows of their H_q + H_kv heads: the
// rotation is read once for all of them, and the next rows are on their way while one is
// worked on.
//
// Bound by HBM: 336 MB (16384 tokens of 40 heads of 128) in 57 us are 5.9 TB/s, 89 % of the
// measured copy rate.  With what rounds exactly left out it took 55 us; with the doubtful
// roundings in a function of their own, through local memory, 63; with the rows
// loaded into registers four at a time 69.  Where a row's 16-byte pieces are paired so that one
// load takes half of each 32-byte sector (adjacent pairs, heads of 64) 24 us became 20.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kRopeResident)
    rope_packed_kernel(const __grid_constant__ RopePackedParams p) {
  constexpr int kLanes = D / 16;
  constexpr int kSlots = kRopeThreads / kLanes;
  __shared__ uint4 ring[kRopeAhead][2][kRopeThreads];
  const int c = threadIdx.x % kLanes;
  allow_later();
  wait_for_earlier();
  const long long t = (long long)blockIdx.x * kSlots + threadIdx.x / kLanes;
  if (t >= p.T) return;
  const int pairs = p.rot_dim / 2, turning = p.rot_dim / 16;
  // the lane's elements lo .. lo + 7 and hi .. hi + 7, such that neighbouring lanes' lie
  // side by side; whether each eight hold pairs that are rotated, and the first pair of
  // the lane's first and second four
  int lo = 8 * c, hi = D / 2 + 8 * c, d[2] = {4 * c, D / 4 + 4 * c};
  bool rotates[2] = {lo < p.rot_dim, hi < p.rot_dim};
  if constexpr (!kInterleaved) {
    rotates[0] = rotates[1] = c < turning;
    d[0] = 8 * c, d[1] = 8 * c + 4;
    hi = pairs + 8 * c;
    if (c >= turning) {
      lo = p.rot_dim + 8 * (c - turning);
      hi = lo + (D - p.rot_dim) / 2;
    }
  }
  // heads [r0, r1) of the queries and the keys behind them; a lane takes what it
  // requested itself
  const int r0 = blockIdx.y * p.rows, r1 = min(r0 + p.rows, p.H_q + p.H_kv);
  int next = r0, put_in = 0;
  const auto request = [&]() {
    if (next < r1) {
      const uint16_t* const src = next < p.H_q ? p.q + t * p.q_st + next * p.q_sh
                                               : p.k + t * p.k_st + (next - p.H_q) * p.k_sh;
      copy_async16(&ring[put_in][0][threadIdx.x], src + lo);
      copy_async16(&ring[put_in][1][threadIdx.x], src + hi);
      ++next;
      put_in = put_in + 1 == kRopeAhead ? 0 : put_in + 1;
    }
    copy_async_commit();
  };
#pragma unroll 1
  for (int n = 0; n < kRopeAhead; ++n) request();   // (needs no position)
  int row[4];
  bool good = true;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    row[a] = a < p.axes ? p.positions[(long long)a * p.T + t] : 0;
    good = good && (unsigned)row[a] < (unsigned)p.rope_rows;
  }
  if (!good) {
    g_packed_status = ATTN_ERR_BAD_INDEX;
    copy_async_wait<0>();
    return;
  }
  uint64_t cs[4] = {}, sn[4] = {};   // cosines and sines of the lane's eight pairs
  const auto row_of = [&](int n) {   // the row that pair n takes
    return n < p.ends[0] ? row[0] : n < p.ends[1] ? row[1] : n < p.ends[2] ? row[2] : row[3];
  };
  const float sign = p.inverse ? -1.f : 1.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // four pairs, of one row as a rule
    if (!rotates[i]) continue;
    int at[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) at[n] = row_of(d[i] + n);
    const auto table = [&](const float* x) {
      const float* const y = x + d[i];
      if (at[0] == at[1] && at[0] == at[2] && at[0] == at[3])
        return *reinterpret_cast<const float4*>(y + (long long)at[0] * pairs);
      return make_float4(y[(long long)at[0] * pairs], y[(long long)at[1] * pairs + 1],
                         y[(long long)at[2] * pairs + 2], y[(long long)at[3] * pairs + 3]);
    };
    const float4 a = table(p.cos), b = table(p.sin);
    cs[2 * i] = f2_pack(a.x, a.y), cs[2 * i + 1] = f2_pack(a.z, a.w);
    sn[2 * i] = f2_pack(sign * b.x, sign * b.y), sn[2 * i + 1] = f2_pack(sign * b.z, sign * b.w);
  }
  int take_from = 0;
#pragma unroll 1
  for (int h = r0; h < r1; ++h) {
    copy_async_wait<kRopeAhead - 1>();
    uint4 w[2] = {ring[take_from][0][threadIdx.x], ring[take_from][1][threadIdx.x]};
    take_from = take_from + 1 == kRopeAhead ? 0 : take_from + 1;
    request();
    if constexpr (kInterleaved) {
      if (rotates[0]) rotate_lane<true>(w[0], {cs[0], cs[1]}, {sn[0], sn[1]});
      if (rotates[1]) rotate_lane<true>(w[1], {cs[2], cs[3]}, {sn[2], sn[3]});
    } else if (rotates[0]) {
      uint4 x = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
      uint4 y = make_uint4(w[0].z, w[0].w, w[1].z, w[1].w);
      rotate_lane<false>(x, {cs[0], cs[1]}, {sn[0], sn[1]});
      rotate_lane<false>(y, {cs[2], cs[3]}, {sn[2], sn[3]});
      w[0] = make_uint4(x.x, x.y, y.x, y.y);
      w[1] = make_uint4(x.z, x.w, y.z, y.w);
    }
    uint16_t* const dst = h < p.H_q ? p.q_out + t * p.qo_st + h * p.qo_sh
                                    : p.k_out + t * p.ko_st + (h - p.H_q) * p.ko_sh;
    *reinterpret_cast<uint4*>(dst + lo) = w[0];
    *reinterpret_cast<uint4*>(dst + hi) = w[1];
  }
}

template <int D>
cudaError_t launch_rope_d(const RopePackedParams& in, bool interleaved, cudaStream_t stream) {
  RopePackedParams p = in;
  const int slots = kRopeThreads / (D / 16);
  const int heads = p.H_q + p.H_kv;
  const long long groups = ((long long)p.T + slots - 1) / slots;
  // A token's heads are shared out so that all thread blocks run at once where they can,
  // and otherwise come in two waves at least (16384 tokens of 40 heads of 128: 57 us,
  // in 1.1 waves 63-65; 9001 tokens of 32 heads of 64 in one wave 15.4 us, in two 17-18).
  long long parts = groups <= kRopeWave ? kRopeWave / groups : (2 * kRopeWave + groups - 1) / groups;
  if (parts > heads) parts = heads;
  p.rows = (int)((heads + parts - 1) / parts);
  const dim3 grid((unsigned)groups, (unsigned)((heads + p.rows - 1) / p.rows));
  return interleaved ? launch_ahead(rope_packed_kernel<D, true>, grid, kRopeThreads, 0, stream, p)
                     : launch_ahead(rope_packed_kernel<D, false>, grid, kRopeThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_packed_plan(const PackedPlan& p, cudaStream_t stream) {
  return launch_ahead(packed_plan_kernel, dim3(1), kPlanThreads, 0, stream, p);
}

cudaError_t launch_rope_packed(const RopePackedParams& p, int D, bool interleaved,
                               cudaStream_t stream) {
  if (D == 128) return launch_rope_d<128>(p, interleaved, stream);
  if (D == 64) return launch_rope_d<64>(p, interleaved, stream);
  return cudaErrorInvalidValue;
}

cudaError_t read_packed_status(int* status, bool reset) {
  cudaError_t err = cudaMemcpyFromSymbol(status, g_packed_status, sizeof(int));
  if (err != cudaSuccess) return err;
  if (reset) {
    const int zero = 0;
    err = cudaMemcpyToSymbol(g_packed_status, &zero, sizeof(int));
  }
  return err;
}

}  // namespace attnpipe
