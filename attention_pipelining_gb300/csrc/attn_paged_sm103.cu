// attn_paged_sm103.cu -- attention of a few query tokens per sequence over a
// paged key/value cache (bf16 or 4-bit), for sm_103a.
//
// Per query row i and visible key j: s_ij = scale q_i . k_j, O_i = sum_j
// exp(s_ij) v_j / sum_j exp(s_ij), in one pass over the keys with a running
// maximum and sum.  A call reads every cached byte once and does 2 (H_q / H_kv)
// S_q multiply-adds per cached element, a handful: it is bound by HBM, and for
// a 4-bit cache next by the instructions that unpack the codes.
//
// One warp takes 16 keys at a time.  The products run on m16n8k16 tensor-core
// instructions, whose fragments come straight from the cache's own order of
// elements (attn_paged.h), with no transposition in between:
//   S = Q K^T    rows are queries (16 to a tile), columns 8 keys: lane (g, t)
//                of the warp (lane = 4 g + t) holds key g's elements as the B
//                fragment and gets S of query row g for keys 2t, 2t + 1;
//   O^T = V^T P^T  rows are elements of v, columns 8 query rows: S's layout is
//                the B fragment of P^T as it stands, and V's pairs of
//                neighbouring keys are the A fragment.
// 4-bit codes enter the products as exact fp16 numbers: a code's four bits are
// put into the mantissa of 256 or of 16, which gives 256 + c or 16 + c in
// one shift and one logic instruction per two elements.  For K the constants
// (and the codes' offset of 8) are taken off by starting the accumulator at
// minus their product with q; K's scales multiply the 32-element partial sums.
// For V they are subtracted; V's scales multiply the probabilities.
//
// Work is dealt out in units of kUnit keys of one (sequence, KV head, tile of
// ROWS query rows): CTA c of G takes units [U c / G, U (c + 1) / G) of all U.
// An item (the units of one sequence, head and row tile) that lies within one
// CTA's range is finished there; otherwise each CTA writes its part to the
// workspace and paged_combine_kernel merges them.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda_fp16.h>

#include "attn_internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace attnpipe {

__device__ int g_paged_status = 0;

namespace {

constexpr int kPgWarps = 4;
constexpr int kPgThreads = kPgWarps * 32;
constexpr int kUnit = 128;                 // keys per unit of work
constexpr uint32_t kFull = 0xffffffffu;
// The reference of a row's exponentials starts below every finite score, and
// far enough above minus infinity that a masked score (-inf) minus it is -inf.
constexpr float kNoMax = -3.0e38f;
// The reference follows the running maximum lazily: it moves only when a
// probability times the largest value scale would pass 2^15 (fp16 holds up
// to 65504), and is then set so that the largest one is 2^6 at most: 2^9 of
// growth before the next move, and values down to 2^-14 (2^-20 of the largest)
// keep all their bits.
constexpr float kMaxProb = 32768.f;
constexpr float kTargetLog2 = 6.f;
// value scales are taken as at least this when the reference is set, so that
// the sum of the probabilities stays finite
constexpr float kMinScale = 5.42101086e-20f;  // 2^-64
constexpr float kMaxSum = 1.0e30f;

// sequences' units: thread i sums those of sequences [i per, (i + 1) per)
struct Plan {
  long long prefix[kPgThreads + 1];
};

__device__ __forceinline__ int clamp_len(const PagedParams& p, int b) {
  const int L = p.lens[b];
  return L < 0 ? 0 : L > p.cache.capacity ? p.cache.capacity : L;
}

// Units of sequence b per (head, row tile): at least one, so that a sequence
// without keys has its rows written too.
__device__ __forceinline__ int units_of(int len) {
  return len <= kUnit ? 1 : (len + kUnit - 1) / kUnit;
}

// Fills the plan; returns the total of the sequences' units.  All threads.
__device__ __forceinline__ long long make_plan(const PagedParams& p, Plan& plan) {
  const int per = (p.cache.B + kPgThreads - 1) / kPgThreads;
  const int b0 = threadIdx.x * per;
  long long sum = 0;
  for (int i = 0; i < per; ++i)
    if (b0 + i < p.cache.B) sum += units_of(clamp_len(p, b0 + i));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += o;
  }
  __shared__ long long warp_sum[kPgWarps];
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) incl += warp_sum[w];
  plan.prefix[threadIdx.x + 1] = incl;
  if (threadIdx.x == 0) plan.prefix[0] = 0;
  __syncthreads();
  return plan.prefix[kPgThreads];
}

// The sequence whose units hold unit v (of the sequences' units, one head and
// row tile), and the number of units before that sequence.
__device__ __forceinline__ int find_sequence(const PagedParams& p, const Plan& plan, long long v,
                                             long long& before) {
  int lo = 0, hi = kPgThreads;   // prefix[lo] <= v < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (plan.prefix[mid] <= v) lo = mid; else hi = mid;
  }
  const int per = (p.cache.B + kPgThreads - 1) / kPgThreads;
  int b = lo * per;
  before = plan.prefix[lo];
  while (true) {
    const int n = units_of(clamp_len(p, b));
    if (before + n > v) return b;
    before += n;
    ++b;
  }
}

// CTAs that take part: no more than there are units, so that none has an
// empty range (the merge reads a part of every CTA between the first and last).
__device__ __forceinline__ int active_ctas(long long U, int ctas) {
  return U < ctas ? (int)U : ctas;
}

// The CTA whose range [U c / G, U (c + 1) / G) holds unit u.
__device__ __forceinline__ int cta_of(long long u, long long U, int G) {
  return (int)(((u + 1) * G - 1) / U);
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

// Each 16-bit half of w holds four codes.  x[n] gets code n of both halves as
// a pair of fp16 numbers base + c: bits 2-5 of the mantissa count in ones
// above 256, bits 6-9 above 16.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&x)[4]) {
  const uint32_t l = w << 2, h = w >> 6;
  x[0] = (l & 0x003c003cu) | 0x5c005c00u;
  x[1] = (l & 0x03c003c0u) | 0x4c004c00u;
  x[2] = (h & 0x003c003cu) | 0x5c005c00u;
  x[3] = (h & 0x03c003c0u) | 0x4c004c00u;
}
constexpr float kBaseEven = 264.f;  // 256 and the codes' offset
constexpr float kBaseOdd = 24.f;    // 16 and the codes' offset

__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// N 32-bit words at p (N = 2 or 4).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}

// scale of key 2t (h = 0) or 2t + 1, group j, from its pair's words
template <int G>
__device__ __forceinline__ float pair_scale(const uint32_t (&w)[G], int h, int j) {
  const uint32_t x = w[h * (G / 2) + (j >> 1)];
  return (j & 1) ? hi_f(x) : lo_f(x);
}

// ---------------------------------------------------------------- one warp

// A warp's running state for one item.  Row r = 16 mt + 8 half + g of the row
// tile belongs to the four lanes of g; mt < MT, half < HALVES.
template <int D, bool kInt4, int ROWS>
struct Warp {
  static constexpr int MT = (ROWS + 15) / 16;        // query tiles of 16 rows
  static constexpr int HALVES = ROWS < 16 ? 1 : 2;   // of which rows 0-7, 8-15 are used
  static constexpr int NR = MT * HALVES;             // rows of a lane
  static constexpr int NT = ROWS / 8;                // column tiles of O^T
  static constexpr int G = D / 32;
  static constexpr int KS = D / 16;                  // k16 steps of Q K^T

  uint32_t q[MT][KS][4];     // A fragments of Q (fp16 or bf16)
  float base[kInt4 ? NR : 1][G];  // what the codes' constants add to S, negated
  float fac[NR];             // S to base-2 exponents
  int lim[NR];               // keys this row sees
  int min_lim;               // keys every row of the tile sees
  float m[NR], l[NR];        // reference and sum
  float o[KS][NT][4];        // O^T

  // The tile's queries, scaled to a power of two around 1 for fp16.
  __device__ __forceinline__ void start(const PagedParams& p, int b, int h, int rt, int len) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int R = p.group * p.S_q;
    int n_q = p.q_lens ? p.q_lens[b] : p.S_q;
    n_q = n_q < 0 ? 0 : n_q > p.S_q ? p.S_q : n_q;
    min_lim = p.causal ? max(0, len - n_q + 1) : len;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int rho = rt * ROWS + mt * 16 + hf * 8 + g;
        const int head = rho / p.S_q, i = rho % p.S_q;
        const bool live = hf < HALVES && rho < R && i < n_q;
        const uint16_t* src = p.q.data + b * p.q.sb + (long long)(h * p.group + head) * p.q.sh +
                              i * p.q.ss;
        uint32_t x[D / 8];   // pairs of this lane's elements
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          // 4-bit: elements 32 c + 8 t ..; bf16: 64 (c / 2) + 8 (2 t + c % 2) ..
          const int d = kInt4 ? 32 * c + 8 * t : 64 * (c >> 1) + 8 * (2 * t + (c & 1));
          const uint4 v = live ? *reinterpret_cast<const uint4*>(src + d) : make_uint4(0, 0, 0, 0);
          x[4 * c] = v.x, x[4 * c + 1] = v.y, x[4 * c + 2] = v.z, x[4 * c + 3] = v.w;
        }
        float f = p.scale_log2;
        if constexpr (kInt4) {
          uint32_t a = 0;
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            a = max(a, max(x[c] & 0x7fffu, (x[c] >> 16) & 0x7fffu));
          a = max(a, __shfl_xor_sync(kFull, a, 1));
          a = max(a, __shfl_xor_sync(kFull, a, 2));
          // 2^e with the row's largest element in [2^e, 2^(e+1)), e in
          // [-126, 126]; elements are taken times 2^-e
          int e = (int)(a >> 7) - 127;
          e = a == 0 ? 0 : e < -126 ? -126 : e > 126 ? 126 : e;
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
          f *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int j = 0; j < G; ++j) {
            float v[8], sum = 0.f;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const uint32_t w = x[4 * j + (n >> 1)];
              v[n] = ((n & 1) ? hi_f(w) : lo_f(w)) * down;
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {   // codes n and n + 4 share a register
              const uint32_t w = pack_f16x2(v[n], v[n + 4]);
              q[mt][2 * j + (n >> 1)][(n & 1) * 2 + hf] = w;
              const __half2 r = *reinterpret_cast<const __half2*>(&w);
              sum += ((n & 1) ? kBaseOdd : kBaseEven) * (__low2float(r) + __high2float(r));
            }
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            if (hf < HALVES) base[mt * HALVES + hf][j] = -sum;
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) q[mt][c >> 1][(c & 1) * 2 + hf] = x[c];
        }
        if (hf < HALVES) {
          const int r = mt * HALVES + hf;
          fac[r] = f;
          lim[r] = !live ? 0 : p.causal ? min(len, max(0, len - n_q + i + 1)) : len;
          m[r] = kNoMax;
          l[r] = 0.f;
        }
      }
#pragma unroll
    for (int d = 0; d < KS; ++d)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[d][n][c] = 0.f;
  }

  // The 16 keys key0 .. key0 + 15, whose K and V blocks lie at kb and vb in
  // shared memory; kMasked where some row may not see all of them.
  template <bool kMasked>
  __device__ __forceinline__ void step(const uint8_t* kb, const uint8_t* vb, int key0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[MT][2][4];   // [query tile][keys 0-7, 8-15]
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      const int key = kt * 8 + g;
      if constexpr (kInt4) {
        uint32_t w[G], sc[G];
        load_words<G>(kb + key * (D / 2) + t * 4 * G, w);
        load_words<G>(kb + 8 * D + (kt * 8 + 2 * t) * 2 * G, sc);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[mt][kt][c] = 0.f;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          uint32_t x[4];
          codes_to_f16(w[j], x);
          const float s0 = pair_scale<G>(sc, 0, j), s1 = pair_scale<G>(sc, 1, j);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float b0 = base[mt * HALVES][j];
            const float b1 = HALVES == 2 ? base[mt * HALVES + HALVES - 1][j] : 0.f;
            float c[4] = {b0, b0, b1, b1};
            mma_f16(c, q[mt][2 * j], x[0], x[1]);
            mma_f16(c, q[mt][2 * j + 1], x[2], x[3]);
            s[mt][kt][0] += c[0] * s0;
            s[mt][kt][1] += c[1] * s1;
            if (HALVES == 2) {
              s[mt][kt][2] += c[2] * s0;
              s[mt][kt][3] += c[3] * s1;
            }
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[mt][kt][c] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[4];
          load_words<4>(kb + 2048 * (c >> 1) + key * 128 + 16 * ((2 * t + (c & 1)) ^ g), w);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_bf16(s[mt][kt], q[mt][2 * c], w[0], w[1]);
            mma_bf16(s[mt][kt], q[mt][2 * c + 1], w[2], w[3]);
          }
        }
      }
    }
    // base-2 exponents where some are masked
    if constexpr (kMasked) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int mt = r / HALVES, hf = r % HALVES;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float& x = s[mt][c >> 1][2 * hf + (c & 1)];
          x *= fac[r];
          if (key0 + (c >> 1) * 8 + 2 * t + (c & 1) >= lim[r]) x = -INFINITY;
        }
      }
    }
    const auto exponent = [&](int r, int c) {   // of row r, key 8 (c / 2) + 2t + c % 2
      const float x = s[r / HALVES][c >> 1][2 * (r % HALVES) + (c & 1)];
      return kMasked ? x : x * fac[r];
    };
    const auto probability = [&](int r, int c) {
      const float x = s[r / HALVES][c >> 1][2 * (r % HALVES) + (c & 1)];
      return ex2_approx(kMasked ? x - m[r] : fmaf(x, fac[r], -m[r]));
    };
    // the values' scales of this lane's keys (pairs 2t, 2t + 1 of each eight)
    uint32_t sv[2][kInt4 ? G : 1];
    float smax = 1.f;
    if constexpr (kInt4) {
      smax = 0.f;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        load_words<G>(vb + 8 * D + (kt * 8 + 2 * t) * 2 * G, sv[kt]);
        if (kMasked) {   // behind the last visible key there may be anything
          const int left = max_lim - key0 - kt * 8 - 2 * t;
#pragma unroll
          for (int j = 0; j < G; ++j)
            if (left <= j / (G / 2)) sv[kt][j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < G; ++j)
          smax = fmaxf(smax, fmaxf(pair_scale<G>(sv[kt], 0, j), pair_scale<G>(sv[kt], 1, j)));
      }
    }
    // probabilities against the lazy reference
    float pr[NR][4];   // [row][keys 2t, 2t + 1, 8 + 2t, 9 + 2t]
    bool over = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float pm = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        pr[r][c] = probability(r, c);
        pm = fmaxf(pm, pr[r][c]);
      }
      over |= pm * smax > kMaxProb || pm > kMaxSum;
    }
    if (__any_sync(kFull, over)) {
      float big = fmaxf(smax, kMinScale);   // (a scale that is a NaN is left out of the maximum)
      big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
      big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
      // log2 of the next power of two
      const float up = (float)((int)(__float_as_uint(big) >> 23) - 126) - kTargetLog2;
      float alpha[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) mx = fmaxf(mx, exponent(r, c));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
        const float next = fmaxf(m[r], mx + up);
        alpha[r] = ex2_approx(m[r] - next);
        m[r] = next;
        l[r] *= alpha[r];
#pragma unroll
        for (int c = 0; c < 4; ++c) pr[r][c] = probability(r, c);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {   // column tile n: rows 8 n + 2t, 8 n + 2t + 1
        const float a0 = __shfl_sync(kFull, alpha[n], 8 * t);
        const float a1 = __shfl_sync(kFull, alpha[n], 8 * t + 4);
#pragma unroll
        for (int d = 0; d < KS; ++d) {
          o[d][n][0] *= a0;
          o[d][n][1] *= a1;
          o[d][n][2] *= a0;
          o[d][n][3] *= a1;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) l[r] += (pr[r][0] + pr[r][1]) + (pr[r][2] + pr[r][3]);
    // O^T += V^T P^T
    if constexpr (kInt4) {
      uint32_t wa[G], wb[G];   // keys 2t, 2t + 1 and 8 + 2t, 9 + 2t: both tokens' words
      load_words<G>(vb + t * (32 * G) + g * (4 * G), wa);
      load_words<G>(vb + (t + 4) * (32 * G) + g * (4 * G), wb);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        uint32_t xa[4], xb[4];
        constexpr int H = G / 2;
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
        codes_to_f16(__byte_perm(wa[j >> 1], wa[H + (j >> 1)], sel), xa);
        codes_to_f16(__byte_perm(wb[j >> 1], wb[H + (j >> 1)], sel), xb);
#pragma unroll
        for (int n = 0; n < 4; ++n) {   // 264 or 24, exactly
          const uint32_t k = (n & 1) ? 0x4e004e00u : 0x5c205c20u;
          xa[n] = h2_sub(xa[n], k);
          xb[n] = h2_sub(xb[n], k);
        }
        const float s0 = pair_scale<G>(sv[0], 0, j), s1 = pair_scale<G>(sv[0], 1, j);
        const float s2 = pair_scale<G>(sv[1], 0, j), s3 = pair_scale<G>(sv[1], 1, j);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float x0 = pr[n][0] * s0, x1 = pr[n][1] * s1, x2 = pr[n][2] * s2, x3 = pr[n][3] * s3;
          if (kMasked) {   // a masked key's scale may be anything
            const int k0 = key0 + 2 * t;
            if (k0 >= lim[n]) x0 = 0.f;
            if (k0 + 1 >= lim[n]) x1 = 0.f;
            if (k0 + 8 >= lim[n]) x2 = 0.f;
            if (k0 + 9 >= lim[n]) x3 = 0.f;
          }
          const uint32_t b0 = pack_f16x2(x0, x1), b1 = pack_f16x2(x2, x3);
          const uint32_t a0[4] = {xa[0], xa[1], xb[0], xb[1]};
          const uint32_t a1[4] = {xa[2], xa[3], xb[2], xb[3]};
          mma_f16(o[2 * j][n], a0, b0, b1);
          mma_f16(o[2 * j + 1][n], a1, b0, b1);
        }
      }
    } else {
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        b0[n] = pack_bf16x2(pr[n][0], pr[n][1]);
        b1[n] = pack_bf16x2(pr[n][2], pr[n][3]);
      }
      // values of keys that no row sees may be anything: keep key pairs
      // by their last visible key
      uint32_t keep0 = kFull, keep1 = kFull;
      if (kMasked) {
        const int left = max_lim - key0 - 2 * t;
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
          const uint32_t a[4] = {__byte_perm(w[0][e], w[1][e], 0x5410u) & keep0,
                                 __byte_perm(w[0][e], w[1][e], 0x7632u) & keep0,
                                 __byte_perm(w[2][e], w[3][e], 0x5410u) & keep1,
                                 __byte_perm(w[2][e], w[3][e], 0x7632u) & keep1};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_bf16(o[4 * sl + e][n], a, b0[n], b1[n]);
        }
      }
    }
  }
  int max_lim;               // keys some row of the tile sees
};

// The first element of v that accumulators o[d][..][0..1] (and [2..3]: the
// next one) hold.
template <bool kInt4>
__device__ __forceinline__ int element_of(int d, int g) {
  return kInt4 ? 32 * (d >> 1) + 4 * g + 2 * (d & 1) : 64 * (d >> 2) + 8 * g + 2 * (d & 3);
}

// Shared memory of a thread block: each warp's ring of kStages stages of 16
// keys (K block, then V block), reused for the merge of the warps' results.
template <int D, bool kInt4, int ROWS>
struct Smem {
  static constexpr int kBlock = kKvBlockBytes<D, kInt4>;
  static constexpr int kStage = 2 * kBlock;
  static constexpr int kStages = kInt4 ? (D == 128 ? 4 : 6) : (D == 128 ? 3 : 4);
  static constexpr int kRing = kStages * kStage;
  static constexpr int kMerge = kPgWarps * ROWS * (D + 4) * 4;
  static constexpr int kBytes = (kPgWarps * kRing > kMerge ? kPgWarps * kRing : kMerge) + 1024;
};

// One warp's stream of 16-key blocks w, w + kPgWarps, .. of a segment through
// its ring: blocks are requested kStages ahead by asynchronous bulk copies
// (4-bit: K's and V's blocks are contiguous, one copy each) or tensor copies
// with the 128-byte swizzle (bf16), and their page numbers one block further.
template <int D, bool kInt4, int ROWS>
struct Stream {
  using S = Smem<D, kInt4, ROWS>;
  uint8_t* ring;
  uint64_t* full;        // [kStages]
  uint32_t issued = 0, taken = 0;   // blocks since the kernel began (all lanes alike)
  uint32_t present = 0;  // bit per stage: the block's page exists
  // the next block to request
  const int* table;
  int left = 0, pg, blk, page;
  long long head;        // 4-bit: byte offset of the head in a page; bf16: the head

  __device__ __forceinline__ void look_up() { page = left > 0 ? table[pg] : -1; }

  __device__ __forceinline__ void begin(const PagedParams& p, int b, int h, int first_block,
                                        int blocks) {
    const KvCache& kc = p.cache;
    table = kc.table + (long long)b * kc.max_blocks;
    left = blocks;
    pg = first_block / kc.blocks_per_page;
    blk = first_block % kc.blocks_per_page;
    head = kInt4 ? (long long)h * kc.blocks_per_page * S::kBlock : h;
    look_up();
  }

  // Requests the next block, if there is one; returns false if its page does
  // not exist.
  __device__ __forceinline__ bool request(const PagedParams& p) {
    if (left <= 0) return true;
    const KvCache& kc = p.cache;
    const uint32_t st = issued % S::kStages;
    const bool ok = (unsigned)page < (unsigned)kc.num_pages;
    if ((threadIdx.x & 31) == 0) {
      uint8_t* dst = ring + st * S::kStage;
      if (ok) {
        mbar_arrive_expect_tx(&full[st], S::kStage);
        if constexpr (kInt4) {
          const long long off = (long long)page * kc.H_kv * kc.blocks_per_page * S::kBlock + head +
                                blk * S::kBlock;
          bulk_load(dst, kc.k + off, S::kBlock, &full[st]);
          bulk_load(dst + S::kBlock, kc.v + off, S::kBlock, &full[st]);
        } else {
          // read once, or once by every row tile
          const uint64_t once = p.row_tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
          const int z = page * kc.H_kv + (int)head;
#pragma unroll
          for (int sl = 0; sl < D / 64; ++sl) {
            tma_load_3d(dst + sl * 2048, &p.tm_k, &full[st], 64 * sl, 16 * blk, z, once);
            tma_load_3d(dst + S::kBlock + sl * 2048, &p.tm_v, &full[st], 64 * sl, 16 * blk, z, once);
          }
        }
      } else {
        mbar_arrive(&full[st]);
      }
    }
    present = (present & ~(1u << st)) | ((uint32_t)ok << st);
    ++issued;
    --left;
    blk += kPgWarps;
    while (blk >= kc.blocks_per_page) {
      blk -= kc.blocks_per_page;
      ++pg;
    }
    look_up();
    return ok;
  }

  // Waits for the oldest requested block; false if the wait ran out of time.
  __device__ __forceinline__ bool take(volatile int* abort_flag, uint64_t budget) {
    const uint32_t st = taken % S::kStages;
    const bool ok = mbar_wait(&full[st], (taken / S::kStages) & 1, abort_flag, budget);
    ++taken;
    return __all_sync(kFull, ok);
  }
};

template <int D, bool kInt4, int ROWS>
__global__ void __launch_bounds__(kPgThreads)
    attn_paged_kernel(const __grid_constant__ PagedParams p) {
  using W = Warp<D, kInt4, ROWS>;
  using S = Smem<D, kInt4, ROWS>;
  extern __shared__ uint8_t smem_raw_pg[];
  uint8_t* smem = align_smem_1024(smem_raw_pg);
  float* sm_o = reinterpret_cast<float*>(smem);   // [kPgWarps][ROWS][D + 4], over the rings
  __shared__ Plan plan;
  __shared__ float sm_m[kPgWarps][ROWS], sm_l[kPgWarps][ROWS];
  __shared__ uint64_t sm_full[kPgWarps][S::kStages];
  __shared__ int sm_abort;
  volatile int* abort_flag = &sm_abort;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const KvCache& kc = p.cache;
  const int HR = kc.H_kv * p.row_tiles;

  if (threadIdx.x < kPgWarps * S::kStages) mbar_init(&sm_full[0][0] + threadIdx.x, 1);
  if (threadIdx.x == 0) sm_abort = 0;
  fence_mbar_init();
  const long long U = make_plan(p, plan) * HR;   // (synchronises the thread block)
  const int G = active_ctas(U, gridDim.x);
  if (blockIdx.x >= G) return;
  const long long u0 = U * blockIdx.x / G, u1 = U * (blockIdx.x + 1) / G;
  long long before;
  int b = find_sequence(p, plan, u0 / HR, before);
  int len = clamp_len(p, b);
  int units = units_of(len);
  int hr = (int)((u0 - before * HR) / units);
  int unit = (int)((u0 - before * HR) % units);
  bool first = true;
  bool bad = p.lens[b] != len;
  Stream<D, kInt4, ROWS> stream;
  stream.ring = smem + warp * S::kRing;
  stream.full = sm_full[warp];

  for (long long u = u0; u < u1;) {
    const int n_units = (int)min((long long)(units - unit), u1 - u);
    const int h = hr / p.row_tiles, rt = hr % p.row_tiles;
    if (p.q_lens && (unsigned)p.q_lens[b] > (unsigned)p.S_q) bad = true;
    W w;
    w.start(p, b, h, rt, len);
    {   // keys some row sees
      int x = 0;
#pragma unroll
      for (int r = 0; r < W::NR; ++r) x = max(x, w.lim[r]);
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) x = max(x, __shfl_xor_sync(kFull, x, d));
      w.max_lim = x;
    }
    const int begin = unit * kUnit, end = min((unit + n_units) * kUnit, w.max_lim);
    const int blocks = end > begin ? (end - begin + 15) / 16 : 0;
    const int mine = (blocks - warp + kPgWarps - 1) / kPgWarps;
    stream.begin(p, b, h, begin / 16 + warp, mine);
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) bad |= !stream.request(p);
#pragma unroll 1
    for (int i = 0, key0 = begin + 16 * warp; i < mine; ++i, key0 += 16 * kPgWarps) {
      const uint32_t st = stream.taken % S::kStages;
      if (!stream.take(abort_flag, p.timeout_ns)) break;
      if ((stream.present >> st) & 1u) {
        const uint8_t* kb = stream.ring + st * S::kStage;
        if (key0 + 16 <= w.min_lim)
          w.template step<false>(kb, kb + S::kBlock, key0);
        else
          w.template step<true>(kb, kb + S::kBlock, key0);
      }
      __syncwarp();
      bad |= !stream.request(p);
    }
    // merge the warps: reference and sum of every row, then O
#pragma unroll
    for (int r = 0; r < W::NR; ++r) {
      float x = w.l[r];
      x += __shfl_xor_sync(kFull, x, 1);
      x += __shfl_xor_sync(kFull, x, 2);
      if (t == 0) {
        sm_m[warp][8 * r + g] = w.m[r];
        sm_l[warp][8 * r + g] = x;
      }
    }
    __syncthreads();
    if (*abort_flag) break;   // (nothing sets it between this barrier and the next take)
#pragma unroll
    for (int n = 0; n < W::NT; ++n) {
      float f[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 8 * n + 2 * t + c;
        float mx = sm_m[0][row];
#pragma unroll
        for (int i = 1; i < kPgWarps; ++i) mx = fmaxf(mx, sm_m[i][row]);
        f[c] = ex2_approx(sm_m[warp][row] - mx);
      }
#pragma unroll
      for (int d = 0; d < W::KS; ++d) {
        float* dst = sm_o + (warp * ROWS + 8 * n + 2 * t) * (D + 4) + element_of<kInt4>(d, g);
        *reinterpret_cast<float2*>(dst) = make_float2(w.o[d][n][0] * f[0], w.o[d][n][2] * f[0]);
        *reinterpret_cast<float2*>(dst + D + 4) =
            make_float2(w.o[d][n][1] * f[1], w.o[d][n][3] * f[1]);
      }
    }
    __syncthreads();
    const bool whole = n_units == units;
    const int slot = 2 * blockIdx.x + (first ? 0 : 1);
    int n_q = p.q_lens ? p.q_lens[b] : p.S_q;
    for (int x = threadIdx.x; x < ROWS * (D / 4); x += kPgThreads) {
      const int row = x / (D / 4), d = 4 * (x % (D / 4));
      const int rho = rt * ROWS + row;
      const int i = rho % p.S_q;
      if (rho >= p.group * p.S_q || i >= n_q) continue;
      float mx = sm_m[0][row];
#pragma unroll
      for (int k = 1; k < kPgWarps; ++k) mx = fmaxf(mx, sm_m[k][row]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kPgWarps; ++k) {
        sum += sm_l[k][row] * ex2_approx(sm_m[k][row] - mx);
        const float4 v = *reinterpret_cast<const float4*>(sm_o + (k * ROWS + row) * (D + 4) + d);
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const float lse2 = sum == 0.f ? -INFINITY : mx + log2f(sum);
      acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
      if (whole) {
        const long long out = (long long)b * p.H_q * p.S_q + (long long)h * p.group * p.S_q + rho;
        *reinterpret_cast<uint2*>(p.o + out * D + d) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        if (d == 0) p.lse[out] = lse2 * 0.6931471805599453f;
      } else {
        const long long out = (long long)slot * ROWS + row;
        *reinterpret_cast<float4*>(p.part_o + out * D + d) = acc;
        if (d == 0) p.part_lse[out] = lse2;
      }
    }
    fence_proxy_async_smem();   // the merge's accesses before the next segment's copies
    __syncthreads();
    u += n_units;
    first = false;
    unit = 0;
    if (++hr == HR && u < u1) {
      hr = 0;
      ++b;
      len = clamp_len(p, b);
      bad = bad || p.lens[b] != len;
      units = units_of(len);
    }
  }
  if (*abort_flag) {
    // a wait ran out: this warp's copies in flight are waited for, once each
    volatile int never = 0;
    while (stream.taken < stream.issued) {
      const uint32_t st = stream.taken % S::kStages;
      mbar_wait(&stream.full[st], (stream.taken / S::kStages) & 1, &never, p.timeout_ns);
      ++stream.taken;
    }
    g_paged_status = ATTN_ERR_TIMEOUT;
    return;
  }
  if (bad) g_paged_status = ATTN_ERR_BAD_INDEX;
}

// Merges the parts of items that several CTAs share: O = sum_c w_c O_c with
// w_c = 2^(lse_c - lse), lse = log2 sum_c 2^lse_c.  One thread block per item.
template <int D, int ROWS>
__global__ void __launch_bounds__(kPgThreads)
    paged_combine_kernel(const __grid_constant__ PagedParams p, int launched) {
  __shared__ Plan plan;
  const KvCache& kc = p.cache;
  const int HR = kc.H_kv * p.row_tiles;
  const long long U = make_plan(p, plan) * HR;
  const int ctas = active_ctas(U, launched);
  const int b = (int)(blockIdx.x / HR), hr = (int)(blockIdx.x % HR);
  const int per = (kc.B + kPgThreads - 1) / kPgThreads;
  long long before = plan.prefix[b / per];
  for (int i = b / per * per; i < b; ++i) before += units_of(clamp_len(p, i));
  const int units = units_of(clamp_len(p, b));
  const long long ub = before * HR + (long long)hr * units;
  const int c0 = cta_of(ub, U, ctas), c1 = cta_of(ub + units - 1, U, ctas);
  if (c0 == c1) return;
  const int slot0 = 2 * c0 + (U * c0 / ctas < ub ? 1 : 0);   // not the first segment of CTA c0
  const int h = hr / p.row_tiles, rt = hr % p.row_tiles;
  const int n_q = p.q_lens ? p.q_lens[b] : p.S_q;
  for (int x = threadIdx.x; x < ROWS * (D / 4); x += kPgThreads) {
    const int row = x / (D / 4), d = 4 * (x % (D / 4));
    const int rho = rt * ROWS + row;
    if (rho >= p.group * p.S_q || rho % p.S_q >= n_q) continue;
    float mx = -INFINITY;
    for (int c = c0; c <= c1; ++c)
      mx = fmaxf(mx, p.part_lse[(long long)(c == c0 ? slot0 : 2 * c) * ROWS + row]);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mx == -INFINITY) mx = 0.f;   // no part sees a key, or all of them are NaN
    for (int c = c0; c <= c1; ++c) {
      const long long at = (long long)(c == c0 ? slot0 : 2 * c) * ROWS + row;
      const float f = ex2_approx(p.part_lse[at] - mx);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * D + d);
      sum += f;
      acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    const long long out = (long long)b * p.H_q * p.S_q + (long long)h * p.group * p.S_q + rho;
    *reinterpret_cast<uint2*>(p.o + out * D + d) =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    if (d == 0)
      p.lse[out] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
  }
}

template <int D, bool kInt4, int ROWS>
cudaError_t launch(const PagedParams& p, cudaStream_t stream) {
  const size_t smem = Smem<D, kInt4, ROWS>::kBytes;
  // per device: the shared-memory attribute set, and the resident CTAs
  static std::atomic<int> resident[64] = {};
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  long long ctas = resident[dev].load(std::memory_order_acquire);
  if (ctas == 0) {
    int sms = 0, per_sm = 0;
    if ((e = cudaFuncSetAttribute(attn_paged_kernel<D, kInt4, ROWS>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
            cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
             &per_sm, attn_paged_kernel<D, kInt4, ROWS>, kPgThreads, smem)) != cudaSuccess)
      return e;
    ctas = (long long)sms * per_sm;
    if (ctas > kPagedMaxCtas) ctas = kPagedMaxCtas;
    if (ctas < 1) return cudaErrorInvalidConfiguration;
    resident[dev].store((int)ctas, std::memory_order_release);
  }
  const long long items = (long long)p.cache.B * p.cache.H_kv * p.row_tiles;
  const long long most = items * ((p.cache.capacity + kUnit - 1) / kUnit);
  if (ctas > most) ctas = most;
  attn_paged_kernel<D, kInt4, ROWS><<<(unsigned)ctas, kPgThreads, smem, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.cache.capacity > kUnit) {   // else every item is one unit: nothing to merge
    paged_combine_kernel<D, ROWS><<<(unsigned)items, kPgThreads, 0, stream>>>(p, (int)ctas);
    e = cudaGetLastError();
  }
  return e;
}

template <int D, bool kInt4>
cudaError_t launch_rows(const PagedParams& p, int rows, cudaStream_t stream) {
  if (rows == 8) return launch<D, kInt4, 8>(p, stream);
  if (rows == 16) return launch<D, kInt4, 16>(p, stream);
  return launch<D, kInt4, 32>(p, stream);
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
