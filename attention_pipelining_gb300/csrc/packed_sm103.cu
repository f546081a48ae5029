// packed_sm103.cu -- packed sequences: the plan of their attention's work, and
// the rotation of queries and keys by positions with several axes
// (include/attn_packed.h).
#include <cstdint>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "kv_cache.cuh"
#include "packed_plan.cuh"
#include "ptx.cuh"
#include "rotate.cuh"

namespace attnpipe {

__device__ int g_packed_status = 0;

namespace {

// ---------------------------------------------------------------- plan

constexpr int kPlanShared = 2048;  // sequences (and one) whose bounds fit shared memory

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Scans of two values at once over the block's threads before this one (0 for the first);
// `warps`: 32 of shared memory (those of warps that the block does not have come last).
template <typename Op>
__device__ __forceinline__ int2 scan_before(int2 x, int2* warps, Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int2 upto = scan_warp(x, op);
  if (lane == 31) warps[warp] = upto;
  __syncthreads();
  if (warp == 0) warps[lane] = scan_warp(warps[lane], op);
  __syncthreads();
  int2 before;
  before.x = __shfl_up_sync(0xffffffffu, upto.x, 1);
  before.y = __shfl_up_sync(0xffffffffu, upto.y, 1);
  if (lane == 0) before = make_int2(0, 0);
  if (warp > 0) before.x = op(warps[warp - 1].x, before.x), before.y = op(warps[warp - 1].y, before.y);
  return before;
}

// Into how many parts an entry of n blocks is cut (see kPackedCtas).
__device__ __forceinline__ int parts_of(int n, int cap) {
  return 2 * n >= 3 * cap ? min((n + cap / 2) / cap, kPackedMostParts) : 1;
}

// One thread block lists the tiles (list 0) and the key blocks (list 1) of all
// sequences, by a counting sort over their costs in blocks (of 128 keys, or of query tiles),
// so that the costliest run first and the last to end are short.  The order among
// equal costs and the parts' slots differ from run to run; no result depends on them.
//
// It stands before every call but the shortest forwards (packed_without_plan), so what
// counts is its latency, a chain of scans with the block's barriers between them: a
// thread takes an entry (found by bisection over the sequences' first entries), and the
// bounds stay in shared memory.  A warp to a sequence, with the bounds read back from
// global memory, took 5 to 9 us, this 3 to 4.  1024 threads, or 512 for up to 31 sequences
// (8 pieces behind prefixes, by itself: 5.8 us, with 1024 6.6; 500 sequences of 1 to 300
// tokens, with the forward: 173.3, with 1024 171.4).
template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PackedPlan p) {
  constexpr int kBuckets = kPlanThreads;   // of costs: a thread to each
  __shared__ int at[2][kBuckets];   // entries of a cost, then where the next of them goes
  __shared__ int2 warps[2][32];
  __shared__ int most[2], slots[2], bounds[4][kPlanShared];
  __shared__ unsigned long long total[2];   // blocks of all entries
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = p.positions, B = p.B, n = B + 1;
  const bool same = p.seq_k == p.seq_q;
  at[0][threadIdx.x] = at[1][threadIdx.x] = 0;
  if (threadIdx.x < 2) most[threadIdx.x] = slots[threadIdx.x] = 0, total[threadIdx.x] = 0;
  // the sequences' first queries and keys, and their first entries in both lists
  const bool fits = n <= kPlanShared;
  int* const q = fits ? bounds[0] : p.seq_q;
  int* const k = same ? q : fits ? bounds[1] : p.seq_k;
  int* const first[2] = {fits ? bounds[2] : p.first[0], fits ? bounds[3] : p.first[1]};
  allow_later();
  // early: behind packed_bwd_prep_kernel, which lets it come when it has itself waited for
  // what is earlier in the stream; its own work the plan neither reads nor changes, and waits
  // for at the end, for those that wait for the plan
  if (!p.early) wait_for_earlier();

#pragma unroll
  for (int i = 0; i < 2; ++i)
    for (int c = threadIdx.x; c < p.n_counters; c += kPlanThreads)
      if (p.counters[i] != nullptr) p.counters[i][c] = 0;

  // The bounds in order, within [0, T]: each the largest up to there.  Then the sequences'
  // first entries, and the most blocks that an entry may have.
  const auto larger = [](int a, int b) { return max(a, b); };
  const auto sum = [](int a, int b) { return a + b; };
  const auto positions = [&](int x) { return packed_over(x, p.over_positions); };
  const auto entries = [&](int queries, int keys) {
    return make_int2(p.tiles != nullptr ? packed_over(queries + 2 * P - 1, p.over_tile) : 0,
                     p.keys != nullptr ? (keys + 127) >> 7 : 0);
  };
  if (n <= 32) {   // (one warp, without the block's barriers: 1 us less)
    if (warp == 0) {
      int2 run;
      if (warp_bounds(p.cu_q, p.cu_k, B, p.T_q, p.T_k, run)) g_packed_status = ATTN_ERR_BAD_INDEX;
      int queries = __shfl_down_sync(0xffffffffu, run.x, 1) - run.x;
      int keys = __shfl_down_sync(0xffffffffu, run.y, 1) - run.y;
      if (lane >= B) queries = keys = 0;
      const int2 e = queries > 0 || keys > 0 ? entries(queries, keys) : make_int2(0, 0);
      const int2 upto = scan_warp(e, sum);
      const int high0 = __reduce_max_sync(0xffffffffu, e.x > 0 ? (keys + 127) >> 7 : 0);
      const int high1 = __reduce_max_sync(0xffffffffu, e.y > 0 ? positions(queries + P - 1) : 0);
      if (lane < n) {
        q[lane] = run.x;
        p.seq_q[lane] = run.x;
        if (!same) k[lane] = run.y;
        first[0][lane] = upto.x - e.x, first[1][lane] = upto.y - e.y;
      }
      if (lane == 0) most[0] = high0, most[1] = high1;
    }
  } else {
    const int per = ceil_div(n, kPlanThreads);
    const int begin = min((int)threadIdx.x * per, n), end = min(begin + per, n);
    int2 run = make_int2(0, 0);
    for (int i = begin; i < end; ++i) {
      run.x = max(run.x, min(p.cu_q[i], p.T_q));
      if (!same) run.y = max(run.y, min(p.cu_k[i], p.T_k));
    }
    run = scan_before(run, warps[0], larger);
    bool bad = false;
    for (int i = begin; i < end; ++i) {
      const int a = p.cu_q[i], b = same ? 0 : p.cu_k[i];
      run.x = max(run.x, min(a, p.T_q));
      run.y = max(run.y, min(b, p.T_k));
      bad |= a != run.x || b != run.y;
      q[i] = run.x;
      p.seq_q[i] = run.x;
      if (!same) k[i] = run.y;
    }
    if (bad) g_packed_status = ATTN_ERR_BAD_INDEX;
    __syncthreads();
    int2 count = make_int2(0, 0), high = make_int2(0, 0);
    for (int b = begin; b < min(end, B); ++b) {
      const int queries = q[b + 1] - q[b], keys = k[b + 1] - k[b];
      const int2 e = entries(queries, keys);
      count.x += e.x, count.y += e.y;
      if (e.x > 0) high.x = max(high.x, (keys + 127) >> 7);
      if (e.y > 0) high.y = max(high.y, positions(queries + P - 1));
    }
    high.x = __reduce_max_sync(0xffffffffu, high.x);
    high.y = __reduce_max_sync(0xffffffffu, high.y);
    if (lane == 0 && high.x > 0) atomicMax(&most[0], high.x);
    if (lane == 0 && high.y > 0) atomicMax(&most[1], high.y);
    run = scan_before(count, warps[1], sum);
    for (int b = begin; b < end; ++b) {
      first[0][b] = run.x, first[1][b] = run.y;
      if (b == B) break;
      const int2 e = entries(q[b + 1] - q[b], k[b + 1] - k[b]);
      run.x += e.x, run.y += e.y;
    }
  }
  __syncthreads();

  // Entry e of either list, whole: its sequence is the last that begins at or before it.
  const auto sequence = [&](int list, int e) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[list][mid] <= e) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  const auto tile_of = [&](int e, PackedTile& x) {
    const int b = sequence(0, e), len = q[b + 1] - q[b], m = k[b + 1] - k[b];
    x = packed_tile_at(b, q[b], len, k[b], m, (e - first[0][b]) * 2 * P, P, p.causal);
    return x.n_blocks;
  };
  // the first query tile that sees a key of block t of a sequence of len queries and m keys
  const auto first_tile = [&](int t, int len, int m) {
    return p.causal ? min(positions(max(t * 128 - (m - len), 0)), positions(len + P - 1)) : 0;
  };
  // (as the first of the group that it is in; the cost is its own)
  const auto keys_of = [&](int e, PackedKeys& x) {
    const int b = sequence(1, e), len = q[b + 1] - q[b], m = k[b + 1] - k[b];
    const int t = e - first[1][b], t0 = t - t % kPackedBand;
    x.k0 = k[b] + t0 * 128;
    x.left = m - t0 * 128;
    x.q0 = q[b];
    x.q_len = len;
    x.vec0 = packed_vec0(q[b], b);
    x.shift = t0 * 128 - (m - len);
    x.size = min((x.left + 127) >> 7, kPackedBand);
    x.before = t - t0;
    x.tiles = positions(len + P - 1);
    x.parts = 1, x.part = 0, x.slot = 0;
    x.first = t0, x.n_work = 0;
    return x.tiles - first_tile(t, len, m);
  };
  // (a thread's first entries stay in registers: there are seldom more)
  PackedTile tile0;
  PackedKeys keys0;
  const int tiles = first[0][B], key_blocks = first[1][B];
  const int tile_cost = (int)threadIdx.x < tiles ? tile_of(threadIdx.x, tile0) : -1;
  const int keys_cost = (int)threadIdx.x < key_blocks ? keys_of(threadIdx.x, keys0) : -1;
  const auto each = [&](auto&& put) {
    if (tile_cost >= 0) put(0, (int)threadIdx.x, tile_cost, &tile0, (PackedKeys*)nullptr);
    if (keys_cost >= 0) put(1, (int)threadIdx.x, keys_cost, (PackedTile*)nullptr, &keys0);
    for (int e = threadIdx.x + kPlanThreads; e < tiles; e += kPlanThreads) {
      PackedTile x;
      const int cost = tile_of(e, x);
      put(0, e, cost, &x, (PackedKeys*)nullptr);
    }
    for (int e = threadIdx.x + kPlanThreads; e < key_blocks; e += kPlanThreads) {
      PackedKeys x;
      const int cost = keys_of(e, x);
      put(1, e, cost, (PackedTile*)nullptr, &x);
    }
  };

  int shift[2], cap[2];
  const bool may_cut =
      2 * most[0] >= 3 * kPackedLeastTile || 2 * most[1] >= 3 * p.least_keys;
  if (may_cut) {
    unsigned long long mine[2] = {0, 0};
    each([&](int list, int, int cost, PackedTile*, PackedKeys*) { mine[list] += cost; });
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
    const unsigned long long least = i == 0 ? kPackedLeastTile : p.least_keys;
    cap[i] = may_cut ? (int)min(max(share, least), 1ull << 29) : 1 << 29;
    shift[i] = 0;
    while ((most[i] >> shift[i]) >= kBuckets) ++shift[i];
  }
  // (where all entries run at once, their order does not matter: one bucket for all)
  const bool sorted = (long long)max(tiles, key_blocks) * p.H_kv > kPackedCtas ||
                      2 * most[0] >= 3 * cap[0] || 2 * most[1] >= 3 * cap[1];
  const auto bucket = [&](int list, int cost) {
    return &at[list][sorted ? kBuckets - 1 - min(cost >> shift[list], kBuckets - 1) : 0];
  };
  // Key blocks, where none is cut, come in groups of up to kPackedBand neighbours, at the
  // first one's cost: the blocks of a group run side by side, one K/V head after the
  // other, and share that head's queries in L2.  (The gradients of 32 heads over 8 of 128,
  // causal, in an earlier build: 16 x 1024 tokens 570 us, in the order of the blocks' own
  // costs, with the heads innermost, 633, in groups of 16 589; 4 x 4096 1417, 1421 and
  // 1450.  Now 522 and 1370.)
  const bool grouped = 2 * most[1] < 3 * cap[1];
  // an entry of n blocks has `parts` parts of `size` blocks, but for the last
  const auto cut = [&](int list, int blocks, int& parts, int& size) {
    parts = parts_of(blocks, cap[list]);
    size = ceil_div(blocks, parts);
    parts = blocks > 0 ? ceil_div(blocks, size) : 1;
  };
  if (sorted) {
    each([&](int list, int, int cost, PackedTile*, PackedKeys* keys) {
      int parts, size;
      if (list == 1 && grouped) {
        if (keys->before == 0) atomicAdd(bucket(1, cost), keys->size);
        return;
      }
      cut(list, cost, parts, size);
      if (parts > 1) atomicAdd(bucket(list, size), parts - 1);
      atomicAdd(bucket(list, cost - (parts - 1) * size), 1);
    });
    __syncthreads();
    // where each cost's entries begin
    const int2 before = scan_before(make_int2(at[0][threadIdx.x], at[1][threadIdx.x]), warps[0], sum);
    at[0][threadIdx.x] = before.x, at[1][threadIdx.x] = before.y;
    __syncthreads();
  }
  if (grouped && p.keys != nullptr) {
    // the groups' places, by their first blocks
    each([&](int list, int e, int cost, PackedTile*, PackedKeys* keys) {
      if (list == 1 && keys->before == 0)
        p.group_at[e] = atomicAdd(bucket(1, cost), keys->size);
    });
    __syncthreads();
  }
  each([&](int list, int e, int cost, PackedTile* tile, PackedKeys* keys) {
    int parts, size;
    if (list == 1 && grouped) {
      p.keys[p.group_at[e - keys->before] + keys->before] = *keys;
      return;
    }
    cut(list, cost, parts, size);
    const int slot = parts > 1 ? atomicAdd(&slots[list], parts) : 0;
    int begins = 0;
    if (list == 1) {   // a group of its own; without a mask each block begins with another
      const int t = keys->before;   // tile, so that those that run at once add to different
      const int block = keys->first + t;   // rows of dQ
      keys->k0 += t * 128, keys->left -= t * 128, keys->shift += t * 128;
      keys->size = 1, keys->before = 0;
      begins = p.causal ? keys->tiles - cost : keys->tiles > 0 ? block % keys->tiles : 0;
      keys->first = block;
    }
    for (int part = 0; part < parts; ++part) {
      const int blocks = part + 1 < parts ? size : cost - part * size;
      const int i = atomicAdd(bucket(list, blocks), 1);
      if (list == 0) {
        tile->jb = part * size, tile->n_blocks = blocks;
        tile->parts = parts, tile->part = part, tile->slot = slot;
        p.tiles[i] = *tile;
      } else {
        if (parts > 1) {
          const int t = begins + part * size;
          keys->first = t < keys->tiles ? t : t - keys->tiles, keys->n_work = blocks;
          keys->parts = parts, keys->part = part, keys->slot = slot;
        }
        p.keys[i] = *keys;
      }
    }
  });
  __syncthreads();
  // (behind the last entry of the last bucket, the lists end)
  if (threadIdx.x == 0) {
    const int last = sorted ? kBuckets - 1 : 0;
    p.head->tiles = at[0][last], p.head->key_blocks = at[1][last];
    p.head->q_first = q[0], p.head->q_end = q[B];
    p.head->next[0] = p.head->next[1] = 0;
    p.head->cut = 2 * most[0] >= 3 * cap[0];
  }
  if (p.early) wait_for_earlier();
}

// ---------------------------------------------------------------- rotation

constexpr int kRopeThreads = 128;
constexpr int kRopeAhead = 4;        // rows of a thread under way
constexpr int kRopeResident = 6;     // thread blocks on an SM
constexpr int kRopeWave = kRopeResident * 152;   // of a whole GB300

// A token's vector of one head is a row that D / 16 neighbouring lanes hold, 16
// elements each: eight first and eight second elements of their pairs, or (adjacent
// pairs, or not rotated) eight of either half of the row.  A thread block takes kSlots consecutive
// tokens and goes with all of them through p.rows of their H_q + H_kv heads: the
// rotation is read once for all of them, and the next rows are on their way while one is
// worked on.
//
// Bound by HBM: 336 MB (16384 tokens of 40 heads of 128) in 57 us are 5.9 TB/s, 89 % of the
// measured copy rate (9001 tokens of 32 heads of 64, adjacent pairs: 74 MB, 15.6 us, 71 %; 32
// tokens 2.5 us, a chain of loads).  With what rounds exactly left out it took 55 us; with the doubtful
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
  return p.B < 32 ? launch_ahead(packed_plan_kernel<512>, dim3(1), 512, 0, stream, p)
                  : launch_ahead(packed_plan_kernel<1024>, dim3(1), 1024, 0, stream, p);
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
