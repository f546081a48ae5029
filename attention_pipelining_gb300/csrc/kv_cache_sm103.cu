// kv_cache_sm103.cu -- new tokens into the paged key/value cache (rotation,
// 4-bit quantisation) and cached tokens back into contiguous tensors.
//
// Both kernels stream.  6.8 TB/s of 4 bytes an element (bf16 read and written)
// leave each SM 22 thread-instructions an element, of 2.6 bytes (a 4-bit write)
// 14: an append into 4 bits runs 22 on average.
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "rotate.cuh"

namespace attnpipe {

__device__ int g_kv_status = 0;

namespace {

constexpr int kKvThreads = 256;         // of the read kernel
constexpr int kAppendThreads = 128;
constexpr int kAhead = 3;               // rows of a thread under way in the append kernel
constexpr int kFewTokens = 8;           // of a sequence, in a decoding step
constexpr int kAppendBlocks = 4864;     // 32 blocks on each of 152 SMs, in four rounds

// ---------------------------------------------------------------- 4 bits

// The codes (one word, element n in nibble n) and the scale of this lane's 8
// elements; its group is the four lanes c / 4 * 4 .. + 3.  rint(x / s) without a
// division an element: x and s are bf16 numbers, so x / s either lies on a tie
// k + 1/2 exactly or at least 2^-10 from one; x (1 / s), off by 2^-21 at most,
// rounded to a multiple of 2^-11 is then on the tie in the first case and on
// the right side of it in the second.
__device__ __forceinline__ uint32_t quantise8(const uint4& w, uint32_t row_mask,
                                              uint32_t& scale_bits) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  // the largest magnitude by the bits' order, where a NaN is above infinity
  const uint32_t m2 = __vimax3_u16x2(x[0] & 0x7fff7fffu, x[1] & 0x7fff7fffu,
                                     __vmaxu2(x[2] & 0x7fff7fffu, x[3] & 0x7fff7fffu));
  uint32_t m = max(m2 & 0xffffu, m2 >> 16);
  m = max(m, __shfl_xor_sync(row_mask, m, 1));
  m = max(m, __shfl_xor_sync(row_mask, m, 2));
  if (m >= 0x7f80u) {   // an infinity or a NaN in the group
    scale_bits = 0x7fffu;
    return 0x88888888u;
  }
  // (m / 7 is never nearer than 2^-13 to a tie of its rounding to bf16)
  scale_bits = pack_bf16x2(__uint_as_float(m << 16) * (1.f / 7.f), 0.f) & 0xffffu;
  const float s = __uint_as_float(scale_bits << 16);
  uint32_t u[8];
  if (s >= 1.0e-30f) {
    const float inv = __frcp_rn(s);
    // 6144 + q has steps of 2^-11; with 1.5 * 2^23 + 8 - 6144 more it has steps of
    // 1, and its last bits are rint(q) + 8, ties to even
    const uint64_t inv2 = f2_pack(inv, inv), grid = f2_pack(6144.f, 6144.f);
    const uint64_t whole = f2_pack(12576776.f, 12576776.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t q =
          f2_add(f2_fma(f2_pack(bf16_lo(x[i]), bf16_hi(x[i])), inv2, grid), whole);
      float q0, q1;
      f2_unpack(q, q0, q1);
      u[2 * i] = __float_as_uint(q0);
      u[2 * i + 1] = __float_as_uint(q1);
    }
  } else {   // few or no significant bits left in s: divide, and clamp
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = (i & 1) ? bf16_hi(x[i >> 1]) : bf16_lo(x[i >> 1]);
      const float q = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(v, s)), -7.f), 7.f) : 0.f;
      u[i] = (uint32_t)((int)q + 8);
    }
  }
  const auto low_bytes = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040u), __byte_perm(c, d, 0x0040u), 0x5410u);
  };
  const uint32_t even = low_bytes(u[0], u[2], u[4], u[6]), odd = low_bytes(u[1], u[3], u[5], u[7]);
  return (even & 0x0f0f0f0fu) | (odd & 0x0f0f0f0fu) << 4;
}

// Stores a lane's codes and its group's scale into the block of its token.
// c: the lane's chunk of the row; r: the token's place in the 16-token block.
template <int D>
__device__ __forceinline__ void store4(uint8_t* block, int r, int c, bool value, uint32_t codes,
                                       uint32_t scale_bits) {
  constexpr int G = D / 32;
  const int j = c >> 2, t = c & 3;
  if (value) {
    uint8_t* p = block + (((r >> 1) * 8 + 2 * t) * 2 + (r & 1)) * 2 * G + 2 * j;
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)codes;                   // g = 2 t
    *reinterpret_cast<uint16_t*>(p + 4 * G) = (uint16_t)(codes >> 16);   // g = 2 t + 1
  } else {
    *reinterpret_cast<uint32_t*>(block + r * (D / 2) + (t * G + j) * 4) = codes;
  }
  if (t == 0)
    *reinterpret_cast<uint16_t*>(block + 8 * D + (r * G + j) * 2) = (uint16_t)scale_bits;
}

// ---------------------------------------------------------------- append

// A token's vector of one head is a row that D / 8 neighbouring lanes hold, 8
// elements each: side by side, or, where the lane rotates pairs (d, d + rot_dim /
// 2), four from either side of its pairs (which takes no exchange between lanes
// and half the cosines; a 4-bit key's lanes change to 8 consecutive elements
// afterwards, one word of codes and a quarter of a scale's group, by way of
// shared memory).  A thread block takes kSlots consecutive tokens, one to a row
// of lanes, and goes with all of them through p.rows of their H_q queries, H_kv
// keys and H_kv values: what belongs to the token (its page, its rotation) is
// read once, and neighbouring tokens, which lie side by side in q_out and in the
// cache, are written together.  The next rows are on their way while one is
// worked on.
//
// Measured, 8192 tokens of 32 + 8 heads of 128 (device time): 4 bits, 181 MB,
// 38 us, 4.8 TB/s (70 % of the measured HBM copy rate; 35 us with adjacent pairs),
// bf16, 206 MB, 35.5 us, 5.8 TB/s (86 %; 34.7 us with adjacent pairs).  Bound by
// the instructions of rotation and quantisation together with the rows' latencies.
// In earlier builds it took 54 us with one token to a block or two rows ahead in
// registers, 44 with eight neighbouring elements a lane throughout, and 39 (bf16 38) with
// the exact roundings in a function of their own (rotate.cuh).
template <int D, bool kInt4, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads, 8)
    kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kSlots = kAppendThreads / kLanes;
  const KvCache& kc = p.cache;
  const int c = threadIdx.x % kLanes;
  const uint32_t row_mask = ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
  // (prompts: 8 ragged ones of up to 1021 tokens 11.8 us, against 12.8; where few
  // tokens are appended, the attention over them comes next: see allow_later)
  if (p.S > kFewTokens) allow_later();
  wait_for_earlier();
  const uint32_t token = blockIdx.x * kSlots + threadIdx.x / kLanes;
  if (token >= (uint32_t)(kc.B * p.S)) return;
  const int b = (int)(token / (uint32_t)p.S), i = (int)(token % (uint32_t)p.S);
  if (p.new_lens) {
    const int n = p.new_lens[b];
    if ((unsigned)n > (unsigned)p.S) g_kv_status = ATTN_ERR_BAD_INDEX;
    if (i >= n) return;
  }
  // this block's rows: heads [q0, q1) of the queries, [k0, k1) of the keys and
  // [v0, v1) of the values
  const int r0 = blockIdx.y * p.rows, r1 = r0 + p.rows;
  const int q0 = min(r0, p.H_q), q1 = min(r1, p.H_q);
  const int k0 = min(max(r0 - p.H_q, 0), kc.H_kv), k1 = min(max(r1 - p.H_q, 0), kc.H_kv);
  const int v0 = min(max(r0 - p.H_q - kc.H_kv, 0), kc.H_kv);
  const int v1 = min(max(r1 - p.H_q - kc.H_kv, 0), kc.H_kv);
  const int rot_lanes = p.rot_dim / 8;
  const bool rotates = c < rot_lanes;
  // the lane's elements lo .. lo + 3, hi .. hi + 3 of a query or a key
  const bool apart = !kInterleaved && p.rot_dim > 0;   // (not in every lane, perhaps)
  const int lo = apart && rotates ? 4 * c : 8 * c;
  const int hi = apart && rotates ? p.rot_dim / 2 + 4 * c : 8 * c + 4;
  const auto store = [&](uint16_t* row, const uint4& w, bool in_halves) {
    if (in_halves) {
      *reinterpret_cast<uint2*>(row + lo) = make_uint2(w.x, w.y);
      *reinterpret_cast<uint2*>(row + hi) = make_uint2(w.z, w.w);
    } else {
      *reinterpret_cast<uint4*>(row + 8 * c) = w;
    }
  };
  const auto source = [&](const KvTensor& t, int h) {
    return t.data + b * t.sb + i * t.ss + h * t.sh;
  };
  // The rows in turn come by way of shared memory, kAhead of them requested in
  // advance; a lane takes what it requested itself.
  __shared__ uint4 ring[kAhead][kAppendThreads];
  __shared__ uint4 regroup[kInt4 && !kInterleaved ? kAppendThreads : 1];
  int left = (q1 - q0) + (k1 - k0) + (v1 - v0), at = q1 - q0, kind = 0, put_in = 0, take_from = 0;
  const uint16_t* src = source(p.q, q0) + lo;
  long long step = p.q.sh;
  bool halves = apart;
  const auto request = [&]() {
    if (left > 0) {
      while (at == 0) {   // on to the keys, then to the values
        src = ++kind == 1 ? source(p.k, k0) + lo : source(p.v, v0) + 8 * c;
        step = kind == 1 ? p.k.sh : p.v.sh;
        at = kind == 1 ? k1 - k0 : v1 - v0;
        halves = apart && kind == 1;
      }
      uint2* const dst = reinterpret_cast<uint2*>(&ring[put_in][threadIdx.x]);
      if (halves) {
        copy_async8(dst, src);
        copy_async8(dst + 1, src + (hi - lo));
      } else {
        copy_async16(dst, src);
      }
      src += step;
      --at;
      --left;
      put_in = put_in + 1 == kAhead ? 0 : put_in + 1;
    }
    copy_async_commit();
  };
  const auto take = [&]() {   // the oldest row, and a request for another
    copy_async_wait<kAhead - 1>();
    const uint4 w = ring[take_from][threadIdx.x];
    take_from = take_from + 1 == kAhead ? 0 : take_from + 1;
    request();
    return w;
  };
#pragma unroll 1
  for (int n = 0; n < kAhead; ++n) request();   // (needs neither position nor page)
  const long long pos = (long long)p.start[b] + i;
  const bool good = pos >= 0 && pos < kc.capacity && (p.rot_dim == 0 || pos < p.rope_rows);
  const int page =
      good ? kc.table[(long long)b * kc.max_blocks + (int)pos / kc.page_size] : -1;
  uint64_t cs[2] = {}, sn[2] = {};   // cosines and sines of the lane's pairs
  if (good && rotates) {
    const long long at = pos * (p.rot_dim / 2) + 4 * c;
    const float4 a = *reinterpret_cast<const float4*>(p.cos + at);
    const float4 d = *reinterpret_cast<const float4*>(p.sin + at);
    cs[0] = f2_pack(a.x, a.y), cs[1] = f2_pack(a.z, a.w);
    sn[0] = f2_pack(d.x, d.y), sn[1] = f2_pack(d.z, d.w);
  }
  if ((unsigned)page >= (unsigned)kc.num_pages) {
    g_kv_status = ATTN_ERR_BAD_INDEX;
    copy_async_wait<0>();
    return;
  }
  const int slot = (int)pos % kc.page_size;
  uint16_t* q_dst = p.q_out + (((long long)b * p.H_q + q0) * p.S + i) * D;
  const long long q_dst_step = (long long)p.S * D;
#pragma unroll 1
  for (int h = q0; h < q1; ++h) {
    uint4 w = take();
    if (rotates) rotate_lane<kInterleaved>(w, cs, sn);
    store(q_dst, w, apart);
    q_dst += q_dst_step;
  }
  const long long head_bytes = (long long)kc.blocks_per_page * kKvBlockBytes<D, kInt4>;
  const auto put = [&](uint8_t* block, uint4 w, bool value) {
    if constexpr (kInt4) {
      if (apart && !value) {   // to 8 consecutive elements a lane
        uint4* const row = regroup + (threadIdx.x - c);
        store(reinterpret_cast<uint16_t*>(row), w, true);
        __syncwarp(row_mask);
        w = row[c];
        __syncwarp(row_mask);
      }
      uint32_t scale;
      const uint32_t codes = quantise8(w, row_mask, scale);
      store4<D>(block, slot & 15, c, value, codes, scale);
    } else {
      store(reinterpret_cast<uint16_t*>(block) + (slot & 15) * D, w, apart && !value);
    }
  };
  uint8_t* dst = const_cast<uint8_t*>(kc.k) + kv_block_offset<D, kInt4>(kc, page, k0, slot >> 4);
#pragma unroll 1
  for (int h = k0; h < k1; ++h) {
    uint4 w = take();
    if (rotates) rotate_lane<kInterleaved>(w, cs, sn);
    put(dst, w, false);
    dst += head_bytes;
  }
  dst = const_cast<uint8_t*>(kc.v) + kv_block_offset<D, kInt4>(kc, page, v0, slot >> 4);
#pragma unroll 1
  for (int h = v0; h < v1; ++h) {
    put(dst, take(), true);
    dst += head_bytes;
  }
}

// ---------------------------------------------------------------- read

// One warp copies one 16-token block of one head's keys or values (blockIdx.y
// even or odd): it reads the block's codes 16 bytes a lane, 8 or 4 consecutive
// elements of which go out together (bf16: 16 bytes of a token's vector).
template <int D, bool kInt4>
__global__ void __launch_bounds__(kKvThreads)
    kv_read_kernel(const __grid_constant__ KvReadParams p) {
  const KvCache& kc = p.cache;
  wait_for_earlier();
  const int lane = threadIdx.x & 31;
  const bool value = blockIdx.y & 1;
  const int h = blockIdx.y >> 1;
  // blocks of a sequence that its S positions may touch
  const int per_seq = (p.S + 15) / 16 + (p.start ? 1 : 0);
  const long long unit = (long long)blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  if (unit >= (long long)kc.B * per_seq) return;
  const int b = (int)(unit / per_seq);
  const long long first = p.start ? p.start[b] : 0;
  const int len = p.lens[b];
  if ((len < 0 || len > kc.capacity || first < 0 || first > kc.capacity) && lane == 0)
    g_kv_status = ATTN_ERR_BAD_INDEX;
  const long long lo = first < 0 ? 0 : first;                     // positions [lo, hi)
  long long hi = first + p.S;
  hi = hi < len ? hi : len;
  hi = hi < kc.capacity ? hi : kc.capacity;
  const long long pos0 = (lo / 16 + unit % per_seq) * 16;         // of the block
  if (pos0 >= hi) return;
  const int blk = (int)(pos0 >> 4);
  const int page = kc.table[(long long)b * kc.max_blocks + blk / kc.blocks_per_page];
  if ((unsigned)page >= (unsigned)kc.num_pages) {
    if (lane == 0) g_kv_status = ATTN_ERR_BAD_INDEX;
    return;
  }
  const uint8_t* block = (value ? kc.v : kc.k) +
                         kv_block_offset<D, kInt4>(kc, page, h, blk % kc.blocks_per_page);
  uint16_t* out = (value ? p.v_out : p.k_out) +
                  (((long long)b * kc.H_kv + h) * p.S + (pos0 - first)) * D;   // of token 0
  const auto wanted = [&](int r) { return pos0 + r >= lo && pos0 + r < hi; };
  if constexpr (!kInt4) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int c = lane % kLanes;
    uint4 w[16 / kRows];
#pragma unroll
    for (int n = 0; n < 16 / kRows; ++n)
      w[n] = *reinterpret_cast<const uint4*>(block + (n * kRows + lane / kLanes) * D * 2 + 16 * c);
#pragma unroll
    for (int n = 0; n < 16 / kRows; ++n) {
      const int r = n * kRows + lane / kLanes;
      if (wanted(r)) *reinterpret_cast<uint4*>(out + r * D + 8 * c) = w[n];
    }
  } else {
    constexpr int G = D / 32;
    const auto two = [](uint32_t codes, int n, float s) {   // elements n, n + 1
      return pack_bf16x2((float)((int)((codes >> (4 * n)) & 15u) - 8) * s,
                         (float)((int)((codes >> (4 * n + 4)) & 15u) - 8) * s);
    };
    if (!value) {   // 4 G bytes: key r's words (t, j)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = n * 8 + (lane >> 2), t = lane & 3;
        uint32_t w[G];
        uint16_t sc[G];
        memcpy(w, __builtin_assume_aligned(block + r * (D / 2) + t * 4 * G, 4 * G), 4 * G);
        memcpy(sc, __builtin_assume_aligned(block + 8 * D + r * 2 * G, 2 * G), 2 * G);
        if (!wanted(r)) continue;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const float s = __uint_as_float((uint32_t)sc[j] << 16);
          *reinterpret_cast<uint4*>(out + r * D + 32 * j + 8 * t) =
              make_uint4(two(w[j], 0, s), two(w[j], 2, s), two(w[j], 4, s), two(w[j], 6, s));
        }
      }
    } else {        // 4 G bytes: elements 32 j + 4 g .. of both tokens of a pair
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int pair = n * 4 + (lane >> 3), g = lane & 7;
        uint16_t w[2][G], sc[2][G];
        memcpy(w, __builtin_assume_aligned(block + (pair * 8 + g) * 4 * G, 4 * G), 4 * G);
        memcpy(sc, __builtin_assume_aligned(block + 8 * D + pair * 4 * G, 4 * G), 4 * G);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = 2 * pair + k;
          if (!wanted(r)) continue;
#pragma unroll
          for (int j = 0; j < G; ++j) {
            const float s = __uint_as_float((uint32_t)sc[k][j] << 16);
            *reinterpret_cast<uint2*>(out + r * D + 32 * j + 4 * g) =
                make_uint2(two(w[k][j], 0, s), two(w[k][j], 2, s));
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p0, int D, bool int4, cudaStream_t stream) {
  KvAppendParams p = p0;
  const int slots = kAppendThreads / (D / 8);
  const int rows = p.H_q + 2 * p.cache.H_kv;
  const long long blocks = ((long long)p.cache.B * p.S + slots - 1) / slots;
  // Where there are few tokens, their rows are spread over several blocks (1024
  // blocks of tokens, 48 rows: cut in five 39 us, in three 41, in ten 45; an earlier build)
  const long long spread = (kAppendBlocks + blocks - 1) / blocks;
  p.rows = spread >= rows ? 1 : (int)((rows + spread - 1) / spread);
  const dim3 grid((unsigned)blocks, (unsigned)((rows + p.rows - 1) / p.rows));
  const auto kernel =
      D == 128 ? int4 ? p.interleaved ? kv_append_kernel<128, true, true>
                                      : kv_append_kernel<128, true, false>
                      : p.interleaved ? kv_append_kernel<128, false, true>
                                      : kv_append_kernel<128, false, false>
               : int4 ? p.interleaved ? kv_append_kernel<64, true, true>
                                      : kv_append_kernel<64, true, false>
                      : p.interleaved ? kv_append_kernel<64, false, true>
                                      : kv_append_kernel<64, false, false>;
  return launch_ahead(kernel, grid, kAppendThreads, 0, stream, p);
}

cudaError_t launch_kv_read(const KvReadParams& p, int D, bool int4, cudaStream_t stream) {
  const long long blocks = (long long)p.cache.B * ((p.S + 15) / 16 + (p.start ? 1 : 0));
  const int per = kKvThreads / 32;
  const dim3 grid((unsigned)((blocks + per - 1) / per), (unsigned)(2 * p.cache.H_kv));
  const auto kernel = D == 128 ? int4 ? kv_read_kernel<128, true> : kv_read_kernel<128, false>
                               : int4 ? kv_read_kernel<64, true> : kv_read_kernel<64, false>;
  return launch_ahead(kernel, grid, kKvThreads, 0, stream, p);
}

cudaError_t read_kv_status(int* status, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_kv_status, sizeof(int));
  if (e == cudaSuccess && reset && *status != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_kv_status, &zero, sizeof(int));
  }
  return e;
}

}  // namespace attnpipe
