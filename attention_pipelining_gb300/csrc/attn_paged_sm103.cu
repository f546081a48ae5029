// attn_paged_sm103.cu -- attention of a few query tokens per sequence over a
// paged key/value cache (bf16 or 4-bit), for sm_103a.
//
// Per query row i and visible key j: s_ij = scale q_i . k_j, O_i = sum_j
// exp(s_ij) v_j / sum_j exp(s_ij), in one pass over the keys with a running
// maximum and sum.  A call reads every cached byte once and does 2 (H_q / H_kv)
// S_q multiply-adds per cached element, a handful: it is bound by HBM, and for
// a 4-bit cache next by the instructions that unpack the codes.
//
// The products run on mma.sync tensor-core instructions, whose fragments come
// straight from the cache's own order of elements (attn_paged.h); lane = 4 g + t:
//   S^T = K Q^T      16 keys by 8 query rows: the lane holds the elements of
//                    keys g and g + 8 as the A fragment, those of query row g as
//                    the B fragment, and gets S of keys g, g + 8 for rows 2t,
//                    2t + 1 (whose maximum, sum and mask it keeps);
//   O^T = V^T P^T    16 elements of v by 8 query rows: P^T is S^T's fragment
//                    transposed by movmatrix, V's pairs of neighbouring keys are
//                    the A fragment, and O^T has the rows 2t, 2t + 1 again.
// (tcgen05 would want 128 query rows to a tile; there are (H_q / H_kv) S_q.)
//
// A 4-bit code is put into the mantissa of the fp16 number 1024 or 64 by one
// mask for two codes (and one shift for eight), and a packed subtraction takes
// that number and the codes' offset of 8 exactly: the products see c - 8.  K's
// scales multiply the 32-element partial sums of S, V's the probabilities.  (On
// sm_103a the fp8 forms of mma.sync are run as conversions and fp16 products, so
// codes as e4m3 bytes cost more than this; fp16 subnormals need no
// subtraction, but their products lost bits.)
//
// A thread block is four consumer warps (or eight) and one producer warp.  The
// producer walks the block's share of the work ahead of the consumers and fills a
// ring of stages, with one asynchronous copy per 16-key block of K and of V, each
// requested by its own lane.
//
// Work is dealt out evenly to the CTAs in units of 128 keys (64 of a bf16 cache) of one
// sequence, KV head and tile of query rows (see Deal).  An item (the units of one sequence,
// head and row tile) that lies within one CTA's range is finished there; otherwise
// each CTA writes its part to the workspace and paged_merge_kernel merges them.
//
// Measured (device time, D = 128, 32 query heads over 8 KV heads): 32 sequences
// of 8192 keys, bf16, 1.07 GB: 162 us, 6.6 TB/s, 98 % of the measured HBM copy
// rate; 4 bits, 303 MB: 67 us, 4.5 TB/s (67 %); 131072 keys of one sequence, 4 bits:
// 37 us (60 %).  What bounds 4 bits is latency: 340 warp-instructions for 16 keys (about
// half of them masks, packed subtractions and scales) would fill the issue slots for
// 38 us and the bytes take 45, but with three consumer warps on a scheduler, each in
// one dependent chain from K's products by the exponentials to V's, there is a ready
// warp in 60 % of the cycles only.  About 10 us of a call are the beginning (plan, page
// table and first keys, one after the other: 5 us) and the end (the warps' merge, the
// CTAs' merge: 5 us).
//
// Tiles of 16 rows and more at D = 128 want more registers than the 168 that two
// blocks of five warps leave a thread, and spill (bf16: 124 to 172 bytes stored, 152 to
// 228 loaded; 4 bits: 124 to 156 and 152 to 192).  8 sequences of 4096 keys with 1, 5
// and 16 queries: bf16 27.5, 34.5 and 60.4 us, 4 bits 17.9, 34.4 and 61.2.
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cuda_fp16.h>

#include "attn_internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace attnpipe {

__device__ int g_paged_status = 0;

namespace {

constexpr int kPlanWarps = 4;              // warps that sum up the sequences' weights
constexpr int kPlanThreads = kPlanWarps * 32;
constexpr int kMergeWarps = 8;
constexpr int kManyParts = 8;              // of an item, on average: more warps for its rows
constexpr int kMaxDevices = 64;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kPgBar = 1;             // named barrier of the consumer warps
// The reference of a row's exponentials starts below every finite score, and
// far enough above minus infinity that a masked score (-inf) minus it is -inf.
constexpr float kNoMax = -3.0e38f;
// The reference follows the running maximum lazily: it moves only when a sum of a
// lane's probabilities in a step (times the largest value scale) would pass
// p.max_prob, and then by enough for 7 bits or more of growth before the next move:
// 4 bits: max_prob is 2^15 (fp16 holds up to 65504), and the largest product is set
//   to 2^6 at most: values down to 2^-14 (2^-20 of the largest) keep all their bits;
// bf16: max_prob is 2^-e with 2^e keys or more in the block table's span, and the
//   largest probability is set to 2^-(e + 8) at most, so that all sums of
//   probabilities stay below 1 and those of probabilities times values below the
//   largest value, which fp32 holds.
constexpr float kMaxProbFp16 = 32768.f;
constexpr float kTargetLog2Fp16 = 6.f;
// value scales are taken as at least this when the reference is set, so that
// the sum of the probabilities stays finite
constexpr float kMinScale = 5.42101086e-20f;  // 2^-64
constexpr float kMaxSum = 1.0e30f;

__device__ __forceinline__ int clamp_len(const PagedParams& p, int b) {
  const int L = p.lens[b];
  return L < 0 ? 0 : L > p.cache.capacity ? p.cache.capacity : L;
}

// Queries of sequence b.
__device__ __forceinline__ int query_count(const PagedParams& p, int b) {
  const int n = p.q_lens ? p.q_lens[b] : p.S_q;
  return n < 0 ? 0 : n > p.S_q ? p.S_q : n;
}

// Units of keys of an item of a sequence of that length: at least one, so
// that a sequence without keys has its rows written too.
__device__ __forceinline__ int units_of(const PagedParams& p, int len) {
  return len <= p.unit ? 1 : (len + p.unit - 1) / p.unit;
}

// An item weighs its units and p.item_cost more, about what the beginning and
// the end of an item take (64 ragged sequences, 4 bits, D = 64, with 1, 2 and 4 units of
// 128 keys: 24.7, 22.1, 24.3 us; the same 256 keys hold for bf16 and for D = 128, where
// others were not compared): the positions 0 .. U - 1 of all items' weights, sequence by
// sequence and within it item by item, are dealt out to G CTAs in even
// consecutive ranges.  The first p.item_cost positions of an item do
// nothing: its unit k is position p.item_cost + k.
struct Deal {
  int U, G, q, r;   // CTA c has q positions, or q + 1 where c < r
  __device__ __forceinline__ Deal(int U_, int launched) : U(U_) {
    G = U < launched ? U : launched;
    q = U / G;
    r = U - q * G;
  }
  __device__ __forceinline__ int start(int c) const { return c * q + min(c, r); }
  __device__ __forceinline__ int owner(int u) const {   // the CTA that has position u
    const int big = r * (q + 1);
    return min(u < big ? u / (q + 1) : r + (u - big) / q, G - 1);
  }
};

// The sequences' weights (of one item each), summed: thread i of the first kPlanThreads
// has those of sequences [i per, (i + 1) per).
struct Plan {
  int before[kPlanThreads];     // of the sequences before thread i's, within its warp
  int warp_sum[kPlanWarps];
};

// All threads of the block call it.  Returns the sum over all sequences.
__device__ __forceinline__ int make_plan(const PagedParams& p, Plan& plan) {
  const int per = (p.cache.B + kPlanThreads - 1) / kPlanThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!p.split) {   // every item is one unit: no need to read the lengths first (7.5 -> 7.2 us)
    __syncthreads();
    return p.cache.B * (p.item_cost + 1);
  }
  if (warp < kPlanWarps) {
    const int b0 = threadIdx.x * per;
    int sum = 0;
    for (int i = 0; i < per; ++i)
      if (b0 + i < p.cache.B) sum += p.item_cost + units_of(p, clamp_len(p, b0 + i));
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += o;
    }
    plan.before[threadIdx.x] = incl - sum;
    if (lane == 31) plan.warp_sum[warp] = incl;
  }
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) total += plan.warp_sum[w];
  return total;
}

// The sequence whose weight covers position v of the sequences' weights, and
// the weight before it.  Whole warps.
__device__ __forceinline__ int find_sequence(const PagedParams& p, const Plan& plan, int v,
                                             int& before) {
  if (!p.split) {
    const int b = min(v / (p.item_cost + 1), p.cache.B - 1);
    before = b * (p.item_cost + 1);
    return b;
  }
  int w = 0, base = 0;
#pragma unroll
  for (int i = 0; i < kPlanWarps - 1; ++i) {
    const int next = base + plan.warp_sum[w];
    if (w == i && v >= next) base = next, ++w;
  }
  // the last thread of that warp whose sequences begin at or before v (threads
  // without sequences begin at the end)
  const int mine = base + plan.before[w * 32 + (threadIdx.x & 31)];
  const uint32_t at = __ballot_sync(kFull, mine <= v);
  const int lane = 31 - __clz(at);
  before = __shfl_sync(kFull, mine, lane);
  const int per = (p.cache.B + kPlanThreads - 1) / kPlanThreads;
  int b = min((w * 32 + lane) * per, p.cache.B - 1);
  for (; b + 1 < p.cache.B; ++b) {
    const int n = p.item_cost + units_of(p, clamp_len(p, b));
    if (before + n > v) break;
    before += n;
  }
  return b;
}

// ---------------------------------------------------------------- fragments

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d = a b
__device__ __forceinline__ void mma_f16_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The 8 x 8 matrix of 16-bit elements held two to a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// fp16 pairs c - 8 of the codes c in bits 0-3 (or 4-7) of x's halves: 1024 + c
// less 1032, 64 + c less 72.  The bases 1024 and 64 come with the parameters, so
// that they are registers: as constants they would cost a second logic
// instruction, which takes one constant at most.
struct CodeBase {
  uint32_t low, high;
};
__device__ __forceinline__ uint32_t low_code(uint32_t x, const CodeBase& base) {
  return h2_sub((x & 0x000f000fu) | base.low, 0x64086408u);
}
__device__ __forceinline__ uint32_t high_code(uint32_t x, const CodeBase& base) {
  return h2_sub((x & 0x00f000f0u) | base.high, 0x54805480u);
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// N 32-bit words at p (N = 1, 2 or 4).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// bf16 element j of the words
template <int N>
__device__ __forceinline__ float element(const uint32_t (&w)[N], int j) {
  return (j & 1) ? hi_f(w[j >> 1]) : lo_f(w[j >> 1]);
}

// ---------------------------------------------------------------- one warp

// A warp's running state for WR query rows of one item, row0 and on.  Row
// 8 n + 2t + c of them (n < NT, c < 2) belongs to the eight lanes of t.
template <int D, bool kInt4, int WR>
struct Warp {
  static constexpr int NT = WR / 8;                  // column tiles of S^T and O^T
  static constexpr int G = D / 32;
  static constexpr int KS = D / 16;
  static constexpr int NB = kInt4 && WR == 8 ? 2 : 1;   // 16-key blocks a step
  // bf16 numbers whose sum stands for a probability in the second product of a bf16
  // cache: off by 2^-16 of it with two, by 2^-8 with one.  Two cost a second product, for
  // which tiles of 8 rows have the time while they wait for memory (32 x 8192 keys
  // 160.2 us with one, 160.3 with two), but not the larger ones (8 x 4096 keys, 16 rows
  // 30.9 and 33.2 us, 64 rows 60.3 and 66.5; 8 ragged with 5 queries 23.2 and 25.4).
  static constexpr int kTerms = WR == 8 ? 2 : 1;

  // B fragments of Q (fp16 for a 4-bit cache): [n][32 elements]{two k16 steps}
  uint32_t q[NT][G][4];
  CodeBase code_base;
  float max_prob, lead;      // see kMaxProbFp16; the reference above the maximum (bf16)
  float fac[NT][2];          // S to base-2 exponents
  int lim[NT][2];            // keys the row sees
  int min_lim, max_lim;      // keys every row of the tile sees, and any may see
  float m[NT][2], l[NT][2];  // reference, and this lane's part of the sum
  float o[KS][NT][4];        // O^T

  // The tile's queries; those of a 4-bit cache scaled by a power of two to
  // [1, 2) at their row's largest element, for fp16.
  __device__ __forceinline__ void start(const PagedParams& p, int b, int h, int row0, int len,
                                        int tile_common, int tile_end) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int R = p.group * p.S_q;
    const int n_q = query_count(p, b);
    code_base.low = p.code_base_low;
    code_base.high = p.code_base_high;
    max_prob = kInt4 ? kMaxProbFp16 : p.max_prob;
    lead = p.lead;
    min_lim = tile_common;
    max_lim = tile_end;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // the fragments hold row 8 n + g
      const int rho = row0 + n * 8 + g;
      const int head = rho / p.S_q, i = rho % p.S_q;
      const bool live = rho < R && i < n_q;
      const uint16_t* src = p.q.data + b * p.q.sb + (long long)(h * p.group + head) * p.q.sh +
                            i * p.q.ss;
      uint32_t x[D / 8];   // pairs of this lane's elements
#pragma unroll
      for (int c = 0; c < G; ++c) {
        // 4-bit: elements 32 c + 8 t ..; bf16: 64 (c / 2) + 8 (2 t + c % 2) ..
        const int d = kInt4 ? 32 * c + 8 * t : 64 * (c >> 1) + 8 * (2 * t + (c & 1));
        const uint4 v = live ? *reinterpret_cast<const uint4*>(src + d) : make_uint4(0, 0, 0, 0);
        x[4 * c] = v.x, x[4 * c + 1] = v.y, x[4 * c + 2] = v.z, x[4 * c + 3] = v.w;
      }
      float f = p.scale_log2;
      if constexpr (kInt4) {
        uint32_t a = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) a = max(a, max(x[c] & 0x7fffu, (x[c] >> 16) & 0x7fffu));
        a = max(a, __shfl_xor_sync(kFull, a, 1));
        a = max(a, __shfl_xor_sync(kFull, a, 2));
        // 2^e with the row's largest element in [2^e, 2^(e+1)); e in [-126, 126]
        int e = (int)(a >> 7) - 127;
        e = a == 0 ? 0 : e < -126 ? -126 : e > 126 ? 126 : e;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        f *= __uint_as_float((uint32_t)(127 + e) << 23);
        f = fminf(fmaxf(f, -FLT_MAX), FLT_MAX);   // (a score of 0 stays 0)
        // codes k and k + 4 of a word lie in one register, codes of even k in bits
        // 0-3 of its halves and of odd k in bits 4-7 (k = 2, 3: after a shift)
#pragma unroll
        for (int j = 0; j < G; ++j) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            v[k] = ((k & 1) ? hi_f(x[4 * j + (k >> 1)]) : lo_f(x[4 * j + (k >> 1)])) * down;
#pragma unroll
          for (int k = 0; k < 4; ++k) x[4 * j + k] = pack_f16x2(v[k], v[k + 4]);
        }
      }
#pragma unroll
      for (int c = 0; c < G; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) q[n][c][k] = x[4 * c + k];
      const int see = !live ? 0 : p.causal ? min(len, max(0, len - n_q + i + 1)) : len;
#pragma unroll
      for (int c = 0; c < 2; ++c) {   // this lane keeps rows 8 n + 2t, 8 n + 2t + 1
        fac[n][c] = __shfl_sync(kFull, f, 8 * t + 4 * c);
        lim[n][c] = __shfl_sync(kFull, see, 8 * t + 4 * c);
        m[n][c] = kNoMax;
        l[n][c] = 0.f;
      }
    }
#pragma unroll
    for (int d = 0; d < KS; ++d)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[d][n][c] = 0.f;
  }

  // The 16 NB keys from key0 on, whose K and V blocks lie in turn at `stage` in
  // shared memory; kMasked where some row may not see all of them or a block
  // is missing (bit 2 i of `have`: block i is there).
  template <bool kMasked>
  __device__ __forceinline__ void step(const uint8_t* stage, int key0, uint32_t have) {
    constexpr int kBlock = kKvBlockBytes<D, kInt4>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[NB][NT][4];   // keys g (rows 2t, 2t + 1), g + 8
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint8_t* kb = stage + 2 * i * kBlock;
      if constexpr (kInt4) {
        uint32_t wa[G], wb[G], sa[G / 2], sb[G / 2];
        load_words<G>(kb + g * (D / 2) + t * 4 * G, wa);
        load_words<G>(kb + (g + 8) * (D / 2) + t * 4 * G, wb);
        load_words<G / 2>(kb + 8 * D + g * 2 * G, sa);
        load_words<G / 2>(kb + 8 * D + (g + 8) * 2 * G, sb);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const uint32_t a0[4] = {low_code(wa[j], code_base), low_code(wb[j], code_base),
                                  high_code(wa[j], code_base), high_code(wb[j], code_base)};
          const uint32_t a1[4] = {
              low_code(wa[j] >> 8, code_base), low_code(wb[j] >> 8, code_base),
              high_code(wa[j] >> 8, code_base), high_code(wb[j] >> 8, code_base)};
          const float s0 = element(sa, j), s1 = element(sb, j);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float c[4];
            mma_f16_new(c, a0, q[n][j][0], q[n][j][1]);
            mma_f16(c, a1, q[n][j][2], q[n][j][3]);
            if (j == 0) {
              s[i][n][0] = c[0] * s0, s[i][n][1] = c[1] * s0;
              s[i][n][2] = c[2] * s1, s[i][n][3] = c[3] * s1;
            } else {
              s[i][n][0] += c[0] * s0, s[i][n][1] += c[1] * s0;
              s[i][n][2] += c[2] * s1, s[i][n][3] += c[3] * s1;
            }
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[i][n][c] = 0.f;
#pragma unroll
        for (int c = 0; c < G; ++c) {
          uint32_t wa[4], wb[4];
          const uint8_t* src = kb + 2048 * (c >> 1) + 16 * ((2 * t + (c & 1)) ^ g);
          load_words<4>(src + g * 128, wa);
          load_words<4>(src + (g + 8) * 128, wb);
          const uint32_t a0[4] = {wa[0], wb[0], wa[1], wb[1]}, a1[4] = {wa[2], wb[2], wa[3], wb[3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_bf16(s[i][n], a0, q[n][c][0], q[n][c][1]);
            mma_bf16(s[i][n], a1, q[n][c][2], q[n][c][3]);
          }
        }
      }
    }
    // base-2 exponents where some are masked; element c of s belongs to key
    // 16 i + g + 8 (c / 2) and row 8 n + 2t + c % 2
    const auto seen = [&](int i, int n, int c) {
      return key0 + 16 * i + 8 * (c >> 1) + g < lim[n][c & 1] && ((have >> (2 * i)) & 1u);
    };
    if constexpr (kMasked) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            s[i][n][c] = seen(i, n, c) ? s[i][n][c] * fac[n][c & 1] : -INFINITY;
    }
    const auto exponent = [&](int i, int n, int c) {
      return kMasked ? s[i][n][c] : s[i][n][c] * fac[n][c & 1];
    };
    // the probabilities of rows 8 n + 2t, 8 n + 2t + 1, and their sums, in pairs
    float pr[NB][NT][4], sum[NT][2];
    const auto probabilities = [&](int n) {
      const uint64_t f2 = kMasked ? f2_pack(1.f, 1.f) : f2_pack(fac[n][0], fac[n][1]);
      const uint64_t m2 = f2_pack(-m[n][0], -m[n][1]);
      uint64_t total = 0;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          const uint64_t x = f2_pack(s[i][n][c], s[i][n][c + 1]);
          float x0, x1;
          f2_unpack(kMasked ? f2_add(x, m2) : f2_fma(x, f2, m2), x0, x1);
          pr[i][n][c] = ex2_approx(x0);
          pr[i][n][c + 1] = ex2_approx(x1);
          const uint64_t pair = f2_pack(pr[i][n][c], pr[i][n][c + 1]);
          total = i + c == 0 ? pair : f2_add(total, pair);
        }
      f2_unpack(total, sum[n][0], sum[n][1]);
    };
    // the values' scales of this lane's keys, and the largest
    uint32_t sv[NB][2][kInt4 ? G / 2 : 1];
    float smax = 1.f;
    if constexpr (kInt4) {
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          load_words<G / 2>(stage + (2 * i + 1) * kBlock + 8 * D + (g + 8 * k) * 2 * G, sv[i][k]);
          if (kMasked) {   // behind the last visible key there may be anything
            const bool any = key0 + 16 * i + 8 * k + g < max_lim && ((have >> (2 * i)) & 1u);
#pragma unroll
            for (int j = 0; j < G / 2; ++j) sv[i][k][j] = any ? sv[i][k][j] : 0u;
          }
#pragma unroll
          for (int j = 0; j < G / 2; ++j) top = max_bf16x2(top, sv[i][k][j]);
        }
      smax = fmaxf(lo_f(top), hi_f(top));   // (a NaN scale is left out of the maximum)
    }
    // against the lazy reference
    float most = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      probabilities(n);
      most = fmaxf(most, fmaxf(sum[n][0], sum[n][1]));
    }
    if (__any_sync(kFull, most * smax > max_prob || (kInt4 && most > kMaxSum))) {
      // how far above the maximum: log2 of the next power of two of the largest of the
      // lanes' value scales, less the target
      const auto above = [&](float big) {
        big = fmaxf(big, kMinScale);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, d));
        return (float)((int)(__float_as_uint(big) >> 23) - 126) - kTargetLog2Fp16;
      };
      const float up_all = kInt4 ? above(smax) : lead;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float alpha[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float up = up_all;
          if constexpr (kInt4 && kMasked) {   // of the keys that this row sees
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < G / 2; ++j)
                  top = max_bf16x2(top, seen(i, n, 2 * k + c) ? sv[i][k][j] : 0u);
            up = above(fmaxf(lo_f(top), hi_f(top)));
          }
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < NB; ++i)
            mx = fmaxf(mx, fmaxf(exponent(i, n, c), exponent(i, n, c + 2)));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
          const float next = fmaxf(m[n][c], mx + up);
          alpha[c] = ex2_approx(m[n][c] - next);
          m[n][c] = next;
          l[n][c] *= alpha[c];
        }
#pragma unroll
        for (int d = 0; d < KS; ++d)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[d][n][c] *= alpha[c & 1];
        probabilities(n);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) l[n][0] += sum[n][0], l[n][1] += sum[n][1];
    // O^T += V^T P^T
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint8_t* vb = stage + (2 * i + 1) * kBlock;
      if constexpr (kInt4) {
        uint32_t wa[G], wb[G];   // keys 2t, 2t + 1 and 8 + 2t, 9 + 2t: both tokens' words
        load_words<G>(vb + t * (32 * G) + g * (4 * G), wa);
        load_words<G>(vb + (t + 4) * (32 * G) + g * (4 * G), wb);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          constexpr int H = G / 2;
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
          const uint32_t ca = __byte_perm(wa[j >> 1], wa[H + (j >> 1)], sel);
          const uint32_t cb = __byte_perm(wb[j >> 1], wb[H + (j >> 1)], sel);
          // elements 0, 1 and 2, 3 of both tokens
          const uint32_t a0[4] = {low_code(ca, code_base), high_code(ca, code_base),
                                  low_code(cb, code_base), high_code(cb, code_base)};
          const uint32_t a1[4] = {low_code(ca >> 8, code_base), high_code(ca >> 8, code_base),
                                  low_code(cb >> 8, code_base), high_code(cb >> 8, code_base)};
          const float s0 = element(sv[i][0], j), s1 = element(sv[i][1], j);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float x[4] = {pr[i][n][0] * s0, pr[i][n][1] * s0, pr[i][n][2] * s1, pr[i][n][3] * s1};
            if constexpr (kMasked) {   // a masked key's scale may be anything
#pragma unroll
              for (int c = 0; c < 4; ++c) x[c] = seen(i, n, c) ? x[c] : 0.f;
            }
            const uint32_t b0 = transpose8(pack_f16x2(x[0], x[1]));
            const uint32_t b1 = transpose8(pack_f16x2(x[2], x[3]));
            mma_f16(o[2 * j][n], a0, b0, b1);
            mma_f16(o[2 * j + 1][n], a1, b0, b1);
          }
        }
      } else {
        uint32_t b0[NT][kTerms], b1[NT][kTerms];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float (&x)[4] = pr[i][n];
          const uint32_t p0 = pack_bf16x2(x[0], x[1]), p1 = pack_bf16x2(x[2], x[3]);
          b0[n][0] = transpose8(p0);
          b1[n][0] = transpose8(p1);
          if constexpr (kTerms == 2) {   // and what that leaves (exact in fp32)
            b0[n][1] = transpose8(pack_bf16x2(x[0] - lo_f(p0), x[1] - hi_f(p0)));
            b1[n][1] = transpose8(pack_bf16x2(x[2] - lo_f(p1), x[3] - hi_f(p1)));
          }
        }
        // Values of keys that some row does not see may be anything, and 0 times NaN
        // is NaN: the products take the keys that every row sees (a mask by pairs),
        const int kb0 = key0 + 16 * i;
        uint32_t keep0 = kFull, keep1 = kFull;
        if constexpr (kMasked) {
          const int left = ((have >> (2 * i)) & 1u) ? min_lim - kb0 - 2 * t : 0;
          keep0 = left <= 0 ? 0u : left == 1 ? 0xffffu : kFull;
          keep1 = left <= 8 ? 0u : left == 9 ? 0xffffu : kFull;
        }
#pragma unroll
        for (int sl = 0; sl < D / 64; ++sl) {
          uint32_t w[4][4];   // keys 2t, 2t + 1, 8 + 2t, 9 + 2t: elements 64 sl + 8 g ..
#pragma unroll
          for (int c = 0; c < 4; ++c)
            load_words<4>(vb + 2048 * sl + ((c >> 1) * 8 + 2 * t + (c & 1)) * 128 +
                              16 * (g ^ (2 * t + (c & 1))), w[c]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t a[4] = {__byte_perm(w[0][e], w[1][e], 0x5410u),
                             __byte_perm(w[0][e], w[1][e], 0x7632u),
                             __byte_perm(w[2][e], w[3][e], 0x5410u),
                             __byte_perm(w[2][e], w[3][e], 0x7632u)};
            if constexpr (kMasked) a[0] &= keep0, a[1] &= keep0, a[2] &= keep1, a[3] &= keep1;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int x = 0; x < kTerms; ++x) mma_bf16(o[4 * sl + e][n], a, b0[n][x], b1[n][x]);
          }
        }
        // and the few others (a causal tile's newest) are added one by one.
        if constexpr (kMasked) {
          const int last = ((have >> (2 * i)) & 1u) ? min(max_lim, kb0 + 16) : 0;
#pragma unroll 1
          for (int k = max(min_lim, kb0); k < last; ++k) {
            const int r = k - kb0;   // its probabilities are lane 4 (r % 8) + t's
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float p[2];
#pragma unroll
              for (int c = 0; c < 2; ++c)
                p[c] = __shfl_sync(kFull, r < 8 ? pr[i][n][c] : pr[i][n][c + 2], (r & 7) * 4 + t);
#pragma unroll
              for (int sl = 0; sl < D / 64; ++sl) {
                uint32_t w[4];
                load_words<4>(vb + 2048 * sl + r * 128 + 16 * (g ^ (r & 7)), w);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                  for (int c = 0; c < 2; ++c)
                    if (k < lim[n][c]) {
                      o[4 * sl + e][n][c] = fmaf(p[c], lo_f(w[e]), o[4 * sl + e][n][c]);
                      o[4 * sl + e][n][c + 2] = fmaf(p[c], hi_f(w[e]), o[4 * sl + e][n][c + 2]);
                    }
              }
            }
          }
        }
      }
    }
  }
};

// The first element of v that accumulators o[d][..][0..1] (and [2..3]: the
// next one) hold.
template <bool kInt4>
__device__ __forceinline__ int element_of(int d, int g) {
  return kInt4 ? 32 * (d >> 1) + 4 * g + 2 * (d & 1) : 64 * (d >> 2) + 8 * g + 2 * (d & 3);
}

// The shape of a thread block: its CW consumer warps take RS groups of WR
// query rows, and for each of them CW / RS groups of keys; a ring of kStages stages
// of kBlocks 16-key blocks (K, V, K, ..), in consecutive runs for the key groups;
// and the merge's scratch.
template <int D, bool kInt4, int WR, int RS, int CW>
struct Shape {
  static constexpr int kRows = WR * RS;
  static constexpr int kThreads = 32 * CW;            // consumers
  static constexpr int kGroups = CW / RS;             // key groups
  static constexpr int NB = Warp<D, kInt4, WR>::NB;
  static constexpr int kBlock = kKvBlockBytes<D, kInt4>;
  static constexpr int kBlocks = (kInt4 ? 2 : 1) * CW;   // of a stage
  static constexpr int kMine = kBlocks / kGroups;     // of them a key group's
  static constexpr int kCopies = 2 * kBlocks;         // one a lane
  static constexpr int kStage = kCopies * kBlock;
  static constexpr int kStages =
      CW == 8 ? 2 : kInt4 || (D == 128 && WR == 8) ? 3 : D == 128 ? 2 : 3;
  // whole stages (bf16: 8 ragged sequences with 5 queries 23.3 us with units of 64 keys, 24.7
  // with 128)
  static constexpr int kUnit = 16 * kBlocks;
  // of all O that the key groups put down for the merge, at a time: half where two blocks of
  // an SM have no room for more
  static constexpr int kTurns = CW == 4 && WR == 8 && D == 128 && !kInt4 ? 2 : 1;
  static constexpr int kWidth = D / kTurns;
  static constexpr int kPitch = kWidth + 4;           // floats a row, against bank conflicts
  static constexpr int kMerge = kGroups * kRows * kPitch * 4;
  static constexpr int kBytes = kStages * kStage + kMerge + 1024;
  // thread blocks per SM
  static constexpr int kCtas = CW == 8 ? 1 : WR == 8 && (kInt4 || D == 64) ? 3 : 2;
  static_assert(kCopies <= 32 && kMine % NB == 0 && kUnit >= kPagedUnit, "stage");
};

// A thread block's share of the work, segment by segment (consecutive units
// of one item).  Producer and consumers walk it alike.  The lengths are read
// again at every sequence; should somebody change them meanwhile, the results are
// unspecified, but every index stays within its range (and a wait between
// warps that no longer agree runs out).
struct Segments {
  int x, x1;            // positions left
  int b, len, units, hr;
  int unit, n;          // of the current segment: its first unit and their number
  int cost;             // p.item_cost
  bool bad;

  // The first segment; false if there is none.  Whole warps.
  __device__ __forceinline__ bool begin(const PagedParams& p, const Plan& plan, const Deal& deal,
                                        int HR) {
    cost = p.item_cost;
    x = deal.start(blockIdx.x);
    x1 = deal.start(blockIdx.x + 1);
    int before;
    b = find_sequence(p, plan, x / HR, before);
    take_sequence(p);
    const int local = x - before * HR, weight = units + cost;
    hr = min(local / weight, HR - 1);
    x = before * HR + hr * weight;   // of the item
    unit = max(0, local - hr * weight - cost);
    return fit();
  }
  __device__ __forceinline__ void take_sequence(const PagedParams& p) {
    len = clamp_len(p, b);
    units = units_of(p, len);
    bad = p.lens[b] != len || (p.q_lens && (unsigned)p.q_lens[b] > (unsigned)p.S_q);
  }
  // How much of the item from `unit` on is this CTA's
  __device__ __forceinline__ bool fit() {
    n = min(units, x1 - x - cost) - unit;
    return n > 0;
  }
  __device__ __forceinline__ bool next(const PagedParams& p, int HR) {
    x += units + cost;
    if (x >= x1) return false;
    unit = 0;
    if (++hr == HR) {
      hr = 0;
      if (++b == p.cache.B) return false;
      take_sequence(p);
    }
    return fit();
  }
  // The position of the item's first unit
  __device__ __forceinline__ int first_position() const { return x + cost; }
};

// Keys that some query row of a tile may see: all of the sequence's, but in
// a causal tile of one head's rows only those up to its last query.
template <int ROWS>
__device__ __forceinline__ int tile_keys(const PagedParams& p, int b, int rt, int len) {
  const int n_q = query_count(p, b);
  const int i0 = (int)((long long)rt * ROWS % p.S_q);
  if (i0 + ROWS > p.S_q) return n_q > 0 ? len : 0;   // rows of more than one head
  if (i0 >= n_q) return 0;
  return p.causal ? max(0, min(len, len - n_q + min(i0 + ROWS, n_q))) : len;
}

// Keys that every query row of a tile sees.
template <int ROWS>
__device__ __forceinline__ int common_keys(const PagedParams& p, int b, int rt, int len) {
  const int i0 = (int)((long long)rt * ROWS % p.S_q);
  const int first = i0 + ROWS > p.S_q ? 0 : i0;
  return p.causal ? max(0, min(len, len - query_count(p, b) + first + 1)) : len;
}

// The producer warp: requests every stage of the block's segments in turn, as
// the consumers free them; lane 2 i + v requests block i of K (v = 0) or V, where
// its page exists (bit 2 i of have[stage]).  Returns the stages requested.
template <int D, bool kInt4, int WR, int RS, int CW>
__device__ __forceinline__ uint32_t produce(const PagedParams& p, Segments seg, uint8_t* ring,
                                            uint64_t* full, uint64_t* empty, uint32_t* have,
                                            volatile int* abort_flag) {
  using S = Shape<D, kInt4, WR, RS, CW>;
  const KvCache& kc = p.cache;
  const int lane = threadIdx.x & 31;
  const int HR = kc.H_kv * p.row_tiles;
  // read once, or once by every row tile
  const uint64_t policy = p.row_tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
  const long long page_bytes = (long long)kc.H_kv * kc.blocks_per_page * S::kBlock;
  const uint8_t* pool = (lane & 1) ? kc.v : kc.k;
  uint8_t* dst = ring + lane * S::kBlock;
  // a stage further: this many pages and blocks
  const int step_pg = S::kBlocks / kc.blocks_per_page, step_blk = S::kBlocks % kc.blocks_per_page;
  uint32_t requested = 0, st = 0, phase = 1;
  bool bad = false;
  do {
    const int h = seg.hr / p.row_tiles, rt = seg.hr % p.row_tiles;
    bad |= seg.bad;
    const int* table = kc.table + (long long)seg.b * kc.max_blocks;
    const int end = min((seg.unit + seg.n) * p.unit,
                        tile_keys<S::kRows>(p, seg.b, rt, seg.len));
    const int blocks = lane < S::kCopies ? (end + 15) >> 4 : 0;
    const uint8_t* head = pool + (long long)h * kc.blocks_per_page * S::kBlock;
    int number = seg.unit * (p.unit / 16) + (lane >> 1);   // this lane's block
    int pg = number / kc.blocks_per_page, blk = number % kc.blocks_per_page;
    int page = number < blocks ? table[pg] : -1;
    for (int key0 = seg.unit * p.unit; key0 < end; key0 += 16 * S::kBlocks) {
      const bool want = number < blocks;
      const bool ok = want && (unsigned)page < (unsigned)kc.num_pages;
      bad |= want && !ok;
      const int now_page = page, now_blk = blk;
      number += S::kBlocks;
      pg += step_pg;
      blk += step_blk;
      if (blk >= kc.blocks_per_page) {
        blk -= kc.blocks_per_page;
        ++pg;
      }
      page = number < blocks ? table[pg] : -1;   // of the next stage
      const uint32_t mask = __ballot_sync(kFull, ok);
      const bool drop = requested == (uint32_t)p.fault_drop_stage;   // test of the wait
      // (the first round finds every stage free)
      if (!__all_sync(kFull, mbar_wait(&empty[st], phase, abort_flag, p.timeout_ns)))
        return requested;
      if (lane == 0 && !drop) {
        have[st] = mask;
        if (mask) mbar_arrive_expect_tx(&full[st], __popc(mask) * S::kBlock);
        else mbar_arrive(&full[st]);
      }
      __syncwarp();
      if (ok && !drop) {
        if constexpr (kInt4) {
          bulk_load(dst + st * S::kStage, head + now_page * page_bytes + now_blk * S::kBlock,
                    S::kBlock, &full[st]);
        } else {
#pragma unroll
          for (int sl = 0; sl < D / 64; ++sl)
            tma_load_3d(dst + st * S::kStage + sl * 2048, (lane & 1) ? &p.tm_v : &p.tm_k, &full[st],
                        64 * sl, 16 * now_blk, now_page * kc.H_kv + h, policy);
        }
      }
      ++requested;
      if (++st == S::kStages) st = 0, phase ^= 1;
    }
  } while (seg.next(p, HR));
  // (never in place of a timeout, which says more: the outputs are then unspecified)
  if (bad) atomicCAS(&g_paged_status, 0, ATTN_ERR_BAD_INDEX);
  // stay until the consumers have had the last stages, and with them every copy
  for (int n = 0; n < S::kStages; ++n) {
    if (requested + n >= S::kStages)
      if (!__all_sync(kFull, mbar_wait(&empty[st], phase, abort_flag, p.timeout_ns))) break;
    if (++st == S::kStages) st = 0, phase ^= 1;
  }
  return requested;
}

template <int D, bool kInt4, int WR, int RS, int CW>
__global__ void __launch_bounds__(32 * CW + 32, Shape<D, kInt4, WR, RS, CW>::kCtas)
    attn_paged_kernel(const __grid_constant__ PagedParams p) {
  using W = Warp<D, kInt4, WR>;
  using S = Shape<D, kInt4, WR, RS, CW>;
  constexpr int ROWS = S::kRows;
  extern __shared__ uint8_t smem_raw_pg[];
  uint8_t* ring = align_smem_1024(smem_raw_pg);
  float* sm_o = reinterpret_cast<float*>(ring + S::kStages * S::kStage);  // [kGroups][ROWS][kPitch]
  __shared__ Plan plan;
  __shared__ float sm_m[S::kGroups][ROWS], sm_l[S::kGroups][ROWS];
  __shared__ uint64_t full[S::kStages], empty[S::kStages];
  __shared__ uint32_t sm_have[S::kStages];
  __shared__ int sm_abort;
  volatile int* abort_flag = &sm_abort;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int HR = p.cache.H_kv * p.row_tiles;

  if (p.split) allow_later();   // the merge kernel may be made ready
  if (threadIdx.x < S::kStages) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], CW);
  }
  fence_mbar_init();
  wait_for_earlier();
  if (threadIdx.x == 0) {
    sm_abort = 0;
    if (p.split && !p.by_item) p.shared[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  const Deal deal(make_plan(p, plan) * HR, gridDim.x);   // (a barrier within)
  if (blockIdx.x >= deal.G) return;
  Segments seg;
  if (!seg.begin(p, plan, deal, HR)) return;

  if (warp == CW) {
    const uint32_t requested =
        produce<D, kInt4, WR, RS, CW>(p, seg, ring, full, empty, sm_have, abort_flag);
    if (*abort_flag) {
      // a wait ran out: the last copies of every stage are waited for, once each
      volatile int never = 0;
      for (uint32_t i = requested > S::kStages ? requested - S::kStages : 0; i < requested; ++i)
        mbar_wait(&full[i % S::kStages], (i / S::kStages) & 1, &never, p.timeout_ns);
      g_paged_status = ATTN_ERR_TIMEOUT;
    }
    return;
  }

  const int rs = warp % RS, kg = warp / RS;
  const uint8_t* mine = ring + kg * S::kMine * 2 * S::kBlock;   // in stage 0
  constexpr uint32_t kAll = 0x55555555u >> (32 - 2 * S::NB);
  uint32_t phase = 0, st = 0;
  do {
    const int h = seg.hr / p.row_tiles, rt = seg.hr % p.row_tiles, b = seg.b;
    const int keys = tile_keys<ROWS>(p, b, rt, seg.len);
    W w;
    w.start(p, b, h, rt * ROWS + rs * WR, seg.len, common_keys<ROWS>(p, b, rt, seg.len), keys);
    const int end = min((seg.unit + seg.n) * p.unit, keys);
    bool ok = true;
#pragma unroll 1
    for (int key0 = seg.unit * p.unit + kg * S::kMine * 16; key0 - kg * S::kMine * 16 < end;
         key0 += 16 * S::kBlocks) {
      ok = __all_sync(kFull, mbar_wait(&full[st], phase, abort_flag, p.timeout_ns));
      if (!ok) break;
      const uint32_t have = sm_have[st] >> (2 * S::kMine * kg);
      const uint8_t* stage = mine + st * S::kStage;
#pragma unroll 1
      for (int i = 0; i < S::kMine; i += S::NB) {
        const int k0 = key0 + 16 * i;
        if (S::kMine > S::NB && k0 >= end) break;
        const uint32_t h2 = have >> (2 * i);
        if (k0 + 16 * S::NB <= w.min_lim && (h2 & kAll) == kAll)
          w.template step<false>(stage + i * 2 * S::kBlock, k0, h2);
        else if (k0 < end)
          w.template step<true>(stage + i * 2 * S::kBlock, k0, h2);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if (++st == S::kStages) st = 0, phase ^= 1;
    }
    // Merge the key groups: every one puts down its rows' references, sums and O, and all
    // threads add them up.  (Two barriers; with O rescaled first and the groups added in
    // halves, four barriers and less shared memory, one sequence of 500 keys took 8.2 us
    // instead of 7.7, 16 x 16 heads x 2048 keys 21.4 instead of 20.7.)
#pragma unroll
    for (int n = 0; n < W::NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = w.l[n][c];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(kFull, x, d);
        if (g == 0) {
          sm_m[kg][rs * WR + 8 * n + 2 * t + c] = w.m[n][c];
          sm_l[kg][rs * WR + 8 * n + 2 * t + c] = x;
        }
      }
    const auto put_down = [&](int turn) {
      float* const mine_o = sm_o + (kg * ROWS + rs * WR) * S::kPitch;
#pragma unroll
      for (int n = 0; n < W::NT; ++n)
#pragma unroll
        for (int d = 0; d < W::KS; ++d)
          if (d / (W::KS / S::kTurns) == turn)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              *reinterpret_cast<float2*>(mine_o + (8 * n + 2 * t + c) * S::kPitch +
                                         element_of<kInt4>(d, g) - turn * S::kWidth) =
                  make_float2(w.o[d][n][c], w.o[d][n][c + 2]);
    };
    put_down(0);
    // (also that every consumer sees whether one of them gave up)
    if (barrier_or(kPgBar, S::kThreads, !ok)) break;
    const bool whole = seg.n == seg.units;
    // a CTA has at most one item that it goes on with and one that goes on
    // after it
    const int slot = 2 * blockIdx.x + (seg.unit == 0 ? 1 : 0);
    if (seg.unit == 0 && threadIdx.x == 0 && (!whole || p.by_item))
      p.shared[p.by_item ? b * HR + seg.hr : blockIdx.x] = make_int4(
          whole ? -1 : b * HR + seg.hr, blockIdx.x, slot,
          whole ? 0 : deal.owner(seg.first_position() + seg.units - 1));
    const int n_q = query_count(p, b);
#pragma unroll
    for (int turn = 0; turn < S::kTurns; ++turn) {
      if (turn > 0) {
        named_barrier_sync(kPgBar, S::kThreads);
        put_down(turn);
        named_barrier_sync(kPgBar, S::kThreads);
      }
      for (int x = threadIdx.x; x < ROWS * (S::kWidth / 4); x += S::kThreads) {
        const int row = x / (S::kWidth / 4), e = 4 * (x % (S::kWidth / 4));
        const int d = turn * S::kWidth + e, rho = rt * ROWS + row;
        if (rho >= p.group * p.S_q || rho % p.S_q >= n_q) continue;
        float mx = sm_m[0][row];
#pragma unroll
        for (int k = 1; k < S::kGroups; ++k) mx = fmaxf(mx, sm_m[k][row]);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < S::kGroups; ++k) {
          const float f = ex2_approx(sm_m[k][row] - mx);
          const float4 v =
              *reinterpret_cast<const float4*>(sm_o + (k * ROWS + row) * S::kPitch + e);
          sum = fmaf(sm_l[k][row], f, sum);
          acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
          acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
        if (whole) {
          const long long out =
              (long long)b * p.H_q * p.S_q + (long long)h * p.group * p.S_q + rho;
          *reinterpret_cast<uint2*>(p.o + out * D + d) =
              make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
          if (d == 0)
            p.lse[out] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
        } else {
          const long long out = (long long)slot * ROWS + row;
          *reinterpret_cast<float4*>(p.part_o + out * D + d) = acc;
          if (d == 0) p.part_lse[out] = sum == 0.f ? -INFINITY : mx + log2f(sum);
        }
      }
    }
    named_barrier_sync(kPgBar, S::kThreads);   // before the scratch is written again
  } while (seg.next(p, HR));
}

// Merges the parts of items that several CTAs share: O = sum_c w_c O_c with
// w_c = 2^(lse_c - lse), lse = log2 sum_c 2^lse_c.  Thread blocks (x, y) merge the
// item that p.shared[x] tells of, if it does: kMergeWarps / kPer rows each, whose
// kPer warps take turns at the parts.  A chain of waits (for the kernel before, the
// entry, the parts, 2.5 to 4 us in all) that moves little data: a warp asks for
// several parts at a time, and where there are many, as few blocks as possible
// come and all of their warps share a row's (8 items of 57 parts: the call takes
// 37.4 us, against 41.0 with blocks for all CTAs and four warps a row).
template <int D, int ROWS, int kPer>
__global__ void __launch_bounds__(32 * kMergeWarps)
    paged_merge_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kRows = kMergeWarps / kPer;
  constexpr int kBatch = kPer > 1 ? 8 : 4;               // parts that a warp loads together
  constexpr int E = D / 32;                              // elements a lane
  // of a part, in the sums: they stay below the largest value (parts are fewer)
  constexpr float kPartShare = 1.f / kPagedMaxCtas;
  __shared__ float sm_acc[kPer > 1 ? kMergeWarps : 1][D], sm_sum[kMergeWarps], sm_max[kMergeWarps];
  wait_for_earlier();
  const int4 it = p.shared[blockIdx.x];
  const int HR = p.cache.H_kv * p.row_tiles, c0 = it.y, parts = it.w - c0 + 1;
  // (an entry is never written where a wait ran out: anything may be there)
  if ((unsigned)it.x >= (unsigned)(p.cache.B * HR) || (unsigned)c0 >= (unsigned)p.ctas ||
      (unsigned)it.w >= (unsigned)p.ctas || (unsigned)(it.z - 2 * c0) > 1u)
    return;
  const int b = it.x / HR, hr = it.x % HR;
  const int h = hr / p.row_tiles, rt = hr % p.row_tiles;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kRows + warp / kPer, share = warp % kPer;
  const int rho = rt * ROWS + row;
  const bool live = rho < p.group * p.S_q && rho % p.S_q < query_count(p, b);
  float mx = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  // adds `share` 2^(l - base) of (s, v) to the sums
  const auto add = [&](float l, float base, float share, float s, const float (&v)[E]) {
    const float f = share * ex2_approx(l - base);
    sum = fmaf(f, s, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, v[e], acc[e]);
  };
  const auto finite = [](float m) { return m == -INFINITY ? 0.f : m; };   // (no part sees a key)
  const auto rescale = [&](float next) {
    const float f = ex2_approx(mx - finite(next));
    sum *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
    mx = next;
  };
  if (live) {
    for (int c = share; c < parts; c += kPer * kBatch) {
      float l[kBatch], v[kBatch][E], next = mx;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int part = c + i * kPer;
        const long long at =   // its place in the workspace
            (long long)(part == 0 ? it.z : 2 * (c0 + part)) * ROWS + row;
        const bool there = part < parts;
        l[i] = there ? p.part_lse[at] : -INFINITY;
        const float* src = p.part_o + at * D + lane * E;
        if constexpr (E == 4) {
          const float4 x = there ? *reinterpret_cast<const float4*>(src) : make_float4(0, 0, 0, 0);
          v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
          const float2 x = there ? *reinterpret_cast<const float2*>(src) : make_float2(0, 0);
          v[i][0] = x.x, v[i][1] = x.y;
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) next = fmaxf(next, l[i]);
      rescale(next);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) add(l[i], finite(mx), kPartShare, 1.f, v[i]);
    }
  }
  if constexpr (kPer > 1) {   // join the row's warps
#pragma unroll
    for (int e = 0; e < E; ++e) sm_acc[warp][lane * E + e] = acc[e];
    if (lane == 0) sm_sum[warp] = sum, sm_max[warp] = mx;
    __syncthreads();
    if (share > 0) return;
    float next = mx;
#pragma unroll
    for (int i = 1; i < kPer; ++i) next = fmaxf(next, sm_max[warp + i]);
    rescale(next);
#pragma unroll
    for (int i = 1; i < kPer; ++i) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = sm_acc[warp + i][lane * E + e];
      add(sm_max[warp + i], finite(mx), 1.f, sm_sum[warp + i], v);
    }
  }
  if (!live) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const long long out = (long long)b * p.H_q * p.S_q + (long long)h * p.group * p.S_q + rho;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + out * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0)
    p.lse[out] = sum == 0.f ? -INFINITY : (mx + log2f(sum / kPartShare)) * 0.6931471805599453f;
}

template <int D, bool kInt4, int WR, int RS, int CW>
cudaError_t launch(const PagedParams& p0, cudaStream_t stream) {
  using S = Shape<D, kInt4, WR, RS, CW>;
  const auto kernel = attn_paged_kernel<D, kInt4, WR, RS, CW>;
  // per device: the shared-memory attribute set, and the resident CTAs
  static std::atomic<int> resident[kMaxDevices] = {};
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  long long ctas = resident[dev].load(std::memory_order_acquire);
  if (ctas == 0) {
    int sms = 0, per_sm = 0;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  S::kBytes)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, S::kThreads + 32,
                                                           S::kBytes)) != cudaSuccess)
      return e;
    ctas = (long long)sms * per_sm;
    if (ctas > kPagedMaxCtas) ctas = kPagedMaxCtas;
    if (ctas < 1) return cudaErrorInvalidConfiguration;
    resident[dev].store((int)ctas, std::memory_order_release);
  }
  PagedParams p = p0;
  p.row_tiles = (int)(((long long)p.group * p.S_q + S::kRows - 1) / S::kRows);
  // Where the block tables span few keys, an item is one unit, which needs no
  // merge kernel and no workspace.  8 items of 250, 500, 1000 keys, 4 bits: 6.0, 7.5,
  // 10.7 us whole, 7.9, 8.9, 9.0 split; bf16 6.9, 9.5, 14.7 and 8.4, 8.6, 8.8; 128 items,
  // 4 bits: 6.5, 7.7, 10.7 and 8.7, 11.0, 12.3; bf16 7.1, 10.3, 15.5 and 10.9, 13.5, 17.3:
  // whole is faster for many items up to the limit, and on the host for all (8.7 us a call
  // against 11.5), but not on the device for a few items near it.  The span decides, since the
  // lengths are on the device: short sequences under a wide table are split.
  const bool split = p.cache.capacity > kPagedWholeKeys;
  p.split = split;
  p.item_cost = kPagedItemKeys / S::kUnit;
  p.unit = split ? S::kUnit : (p.cache.capacity + S::kUnit - 1) / S::kUnit * S::kUnit;
  const long long items = (long long)p.cache.B * p.cache.H_kv * p.row_tiles;
  // positions are counted in an int: larger units where there could be too many
  while (items * ((p.cache.capacity + p.unit - 1) / p.unit + p.item_cost) >= (1ll << 31))
    p.unit *= 2;
  const long long most = items * ((p.cache.capacity + p.unit - 1) / p.unit);
  if (ctas > most) ctas = most;
  p.ctas = (int)ctas;
  p.by_item = split && items * kManyParts <= ctas;
  e = launch_ahead(kernel, dim3((unsigned)ctas), S::kThreads + 32, S::kBytes, stream, p);
  if (e != cudaSuccess || !split) return e;
  const long long rows = (long long)p.group * p.S_q;
  const unsigned live = (unsigned)(rows < S::kRows ? rows : S::kRows);   // of a tile
  // Few items of many parts each: a block for every item and row, whose warps share the
  // parts; else a block for every CTA's item and eight rows, a row to a warp
  if (p.by_item)
    return launch_ahead(paged_merge_kernel<D, S::kRows, kMergeWarps>, dim3((unsigned)items, live),
                        32 * kMergeWarps, 0, stream, p);
  return launch_ahead(paged_merge_kernel<D, S::kRows, 1>,
                      dim3((unsigned)ctas, (live + kMergeWarps - 1) / kMergeWarps),
                      32 * kMergeWarps, 0, stream, p);
}

// SMs of the current device (each device is asked once).
cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  *sms = known[dev].load(std::memory_order_acquire);
  if (*sms > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) known[dev].store(*sms, std::memory_order_release);
  return e;
}

template <int D, bool kInt4>
cudaError_t launch_rows(const PagedParams& p, int rows, cudaStream_t stream) {
  // No more short items than SMs: blocks of eight consumer warps, one on an SM (128 items of
  // 1000 keys, D = 128: 10.7 us, 15.5 in bf16, against 11.5 and 17.0 with blocks of
  // four; 8 items of 500 keys 7.5 and 9.5 against 7.7 and 10.4)
  if (rows == 8 && p.cache.capacity <= kPagedWholeKeys) {
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    if ((long long)p.cache.B * p.cache.H_kv <= sms) return launch<D, kInt4, 8, 1, 8>(p, stream);
  }
  if (rows == 8) return launch<D, kInt4, 8, 1, 4>(p, stream);
  if (rows == 16) return launch<D, kInt4, 16, 1, 4>(p, stream);
  if (rows == 32) return launch<D, kInt4, 16, 2, 4>(p, stream);
  return launch<D, kInt4, 16, 4, 4>(p, stream);
}

}  // namespace

cudaError_t launch_attn_paged(const PagedParams& p, int D, bool int4, int rows,
                              cudaStream_t stream) {
  if (D == 128) return int4 ? launch_rows<128, true>(p, rows, stream)
                            : launch_rows<128, false>(p, rows, stream);
  return int4 ? launch_rows<64, true>(p, rows, stream) : launch_rows<64, false>(p, rows, stream);
}

cudaError_t read_paged_status(int* status, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_paged_status, sizeof(int));
  if (e == cudaSuccess && reset && *status != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int));
  }
  return e;
}

}  // namespace attnpipe
