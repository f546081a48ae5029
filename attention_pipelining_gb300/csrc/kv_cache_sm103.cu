// kv_cache_sm103.cu -- new tokens into the paged key/value cache (rotation,
// 4-bit quantisation) and cached tokens back into contiguous tensors.
//
// Both kernels stream: a token's vector of one head is a "row" of D elements
// that D / 8 neighbouring lanes hold, 16 bytes (8 elements) each, so that one
// lane's 8 elements of a 4-bit row are one 32-bit word of codes and a scale's
// group of 32 elements is four neighbouring lanes.
#include <cstdint>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace attnpipe {

__device__ int g_kv_status = 0;

namespace {

constexpr int kKvThreads = 256;

// ---------------------------------------------------------------- rotation

// x a - y b rounded once to bf16 (returned as a float): the products' and the
// sum's rounding errors are recovered (fma, two-sum) and added back, and the
// fp32 result, when it falls on a tie of the bf16 rounding that the remainder
// breaks, is moved one step to the remainder's side.  x and y are bf16 values
// and a and b fp32, so the exact value has at most 32 significant bits a
// product: without this, about one element in 2^15 would round the other way
// than the exact value, and in a 4-bit cache change its code.  Non-finite
// values take the plain formula's result.
__device__ __forceinline__ float rotate_bf16(float x, float a, float y, float b) {
  const float h = __fmul_rn(x, a), h2 = __fmul_rn(-y, b);
  const float e = __fmaf_rn(x, a, -h), e2 = __fmaf_rn(-y, b, -h2);
  const float s = __fadd_rn(h, h2);
  const float t = __fsub_rn(s, h);
  const float es = __fadd_rn(__fsub_rn(h, __fsub_rn(s, t)), __fsub_rn(h2, t));
  const float lo = __fadd_rn(es, __fadd_rn(e, e2));
  const float r = __fadd_rn(s, lo);
  if (!(fabsf(r) <= 3.4028235e38f)) return s;   // an infinity or a NaN
  const float rem = __fsub_rn(lo, __fsub_rn(r, s));
  uint32_t u = __float_as_uint(r);
  if ((u & 0xffffu) == 0x8000u && rem != 0.f) u += ((rem > 0.f) == (r > 0.f)) ? 1u : 0xffffffffu;
  return __uint_as_float(u);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The rotation of this lane's 8 elements (chunk c of its row), in place;
// every lane of the row takes part.  With pairs (d, d + rot / 2) the partner
// chunk is another lane's; with adjacent pairs it is the lane's own.
template <int kLanes>
__device__ __forceinline__ void rotate_chunk(uint4& w, int c, int rot_chunks, bool interleaved,
                                             const float (&cs)[8], const float (&sn)[8]) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
  if (interleaved) {
    if (c < rot_chunks) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = bf16_lo(x[i]), b = bf16_hi(x[i]);
        x[i] = pack_bf16x2(rotate_bf16(a, cs[i], b, sn[i]), rotate_bf16(b, cs[i], -a, sn[i]));
      }
    }
  } else {
    const int half = rot_chunks >> 1;
    const bool first = c < half;
    const int partner = first ? c + half : c < rot_chunks ? c - half : c;
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner, kLanes);
    if (c < rot_chunks) {
      const float sg = first ? 1.f : -1.f;   // (a cos - b sin), (b cos + a sin)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = pack_bf16x2(
            rotate_bf16(bf16_lo(x[i]), cs[2 * i], sg * bf16_lo(y[i]), sn[2 * i]),
            rotate_bf16(bf16_hi(x[i]), cs[2 * i + 1], sg * bf16_hi(y[i]), sn[2 * i + 1]));
    }
  }
  w = make_uint4(x[0], x[1], x[2], x[3]);
}

// ---------------------------------------------------------------- 4 bits

// The codes (one word, element n in nibble n) and the scale of this lane's 8
// elements; its group is the four lanes c / 4 * 4 .. + 3.  The division is
// the IEEE one: a code on a tie goes to the even one, as the definition says.
__device__ __forceinline__ uint32_t quantise8(const uint4& w, uint32_t& scale_bits) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  // the largest magnitude by the bits' order, where a NaN is above infinity
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (m >= 0x7f80u) {   // an infinity or a NaN in the group
    scale_bits = 0x7fffu;
    return 0x88888888u;
  }
  scale_bits = pack_bf16x2(__fdiv_rn(__uint_as_float(m << 16), 7.f), 0.f) & 0xffffu;
  const float s = __uint_as_float(scale_bits << 16);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = (i & 1) ? bf16_hi(x[i >> 1]) : bf16_lo(x[i >> 1]);
    const float q = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(v, s)), -7.f), 7.f) : 0.f;
    codes |= (uint32_t)((int)q + 8) << (4 * i);
  }
  return codes;
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

template <int D>
__device__ __forceinline__ void load4(const uint8_t* block, int r, int c, bool value,
                                      uint32_t& codes, float& scale) {
  constexpr int G = D / 32;
  const int j = c >> 2, t = c & 3;
  if (value) {
    const uint8_t* p = block + (((r >> 1) * 8 + 2 * t) * 2 + (r & 1)) * 2 * G + 2 * j;
    codes = (uint32_t)*reinterpret_cast<const uint16_t*>(p) |
            (uint32_t)*reinterpret_cast<const uint16_t*>(p + 4 * G) << 16;
  } else {
    codes = *reinterpret_cast<const uint32_t*>(block + r * (D / 2) + (t * G + j) * 4);
  }
  scale = __uint_as_float(
      (uint32_t)*reinterpret_cast<const uint16_t*>(block + 8 * D + (r * G + j) * 2) << 16);
}

// ---------------------------------------------------------------- append

// One thread block handles heads blockIdx.y * kSlots * p.rounds .. of one
// token (its rows: H_q queries, H_kv keys, H_kv values), kSlots at a time: the
// token's rotation, 8 cosines and sines a lane, is read once for all of them.
template <int D, bool kInt4>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const KvAppendParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kSlots = kKvThreads / kLanes;
  const int b = blockIdx.x / p.S, i = blockIdx.x % p.S;
  if (p.new_lens && i >= p.new_lens[b]) return;
  const int c = threadIdx.x % kLanes, slot_row = threadIdx.x / kLanes;
  const long long pos = (long long)p.start[b] + i;
  const KvCache& kc = p.cache;
  const bool in_range = pos >= 0 && pos < kc.capacity && (p.rot_dim == 0 || pos < p.rope_rows);
  int page = -1;
  if (in_range) page = kc.table[(long long)b * kc.max_blocks + pos / kc.page_size];
  if (page < 0 || page >= kc.num_pages) {
    if (threadIdx.x == 0) g_kv_status = ATTN_ERR_BAD_INDEX;
    return;
  }
  const int slot = (int)(pos % kc.page_size);
  const int rot_chunks = p.rot_dim / 8;
  float cs[8], sn[8];
  if (c < rot_chunks) {
    const long long row = pos * (p.rot_dim / 2);
    if (p.interleaved) {
      const float4 a = *reinterpret_cast<const float4*>(p.cos + row + 4 * c);
      const float4 d = *reinterpret_cast<const float4*>(p.sin + row + 4 * c);
      cs[0] = a.x, cs[1] = a.y, cs[2] = a.z, cs[3] = a.w;
      sn[0] = d.x, sn[1] = d.y, sn[2] = d.z, sn[3] = d.w;
    } else {
      const int at = 8 * (c < rot_chunks / 2 ? c : c - rot_chunks / 2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 a = *reinterpret_cast<const float4*>(p.cos + row + at + 4 * h);
        const float4 d = *reinterpret_cast<const float4*>(p.sin + row + at + 4 * h);
        cs[4 * h] = a.x, cs[4 * h + 1] = a.y, cs[4 * h + 2] = a.z, cs[4 * h + 3] = a.w;
        sn[4 * h] = d.x, sn[4 * h + 1] = d.y, sn[4 * h + 2] = d.z, sn[4 * h + 3] = d.w;
      }
    }
  }
  const int rows = p.H_q + 2 * kc.H_kv;
  for (int n = 0; n < p.rounds; ++n) {
    const int row = (blockIdx.y * p.rounds + n) * kSlots + slot_row;
    const bool live = row < rows;
    const bool is_q = row < p.H_q;
    const bool is_v = row >= p.H_q + kc.H_kv;
    const int h = is_q ? row : is_v ? row - p.H_q - kc.H_kv : row - p.H_q;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) {
      const KvTensor& t = is_q ? p.q : is_v ? p.v : p.k;
      w = *reinterpret_cast<const uint4*>(t.data + b * t.sb + h * t.sh + i * t.ss + 8 * c);
    }
    // a row's lanes agree on is_v, but a warp's rows may not: all take part
    uint4 turned = w;
    if (rot_chunks) rotate_chunk<kLanes>(turned, c, rot_chunks, p.interleaved, cs, sn);
    if (!is_v) w = turned;
    uint32_t codes = 0, scale = 0;
    if (kInt4) codes = quantise8(w, scale);
    if (!live) continue;
    if (is_q) {
      *reinterpret_cast<uint4*>(p.q_out + (((long long)b * p.H_q + h) * p.S + i) * D + 8 * c) = w;
    } else {
      uint8_t* block = const_cast<uint8_t*>(is_v ? kc.v : kc.k) +
                       kv_block_offset<D, kInt4>(kc, page, h, slot >> 4);
      if (kInt4)
        store4<D>(block, slot & 15, c, is_v, codes, scale);
      else
        *reinterpret_cast<uint4*>(block + (slot & 15) * D * 2 + 16 * c) = w;
    }
  }
}

// ---------------------------------------------------------------- read

// One row slot handles rows of k_out (blockIdx.y even: keys, odd: values).
template <int D, bool kInt4>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvReadParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kSlots = kKvThreads / kLanes;
  const KvCache& kc = p.cache;
  const int c = threadIdx.x % kLanes;
  const bool value = blockIdx.y & 1;
  const long long row = (long long)blockIdx.x * kSlots + threadIdx.x / kLanes;
  const int h = blockIdx.y >> 1;
  const long long per_head = (long long)kc.B * p.S;
  if (row >= per_head) return;
  const int b = (int)(row / p.S), i = (int)(row % p.S);
  const long long pos = (p.start ? (long long)p.start[b] : 0) + i;
  const int len = p.lens[b];
  if (len < 0 || len > kc.capacity || pos < 0) {
    if (c == 0) g_kv_status = ATTN_ERR_BAD_INDEX;
    if (pos < 0) return;
  }
  if (pos >= len || pos >= kc.capacity) return;
  const int page = kc.table[(long long)b * kc.max_blocks + pos / kc.page_size];
  if (page < 0 || page >= kc.num_pages) {
    if (c == 0) g_kv_status = ATTN_ERR_BAD_INDEX;
    return;
  }
  const int slot = (int)(pos % kc.page_size);
  const uint8_t* block = (value ? kc.v : kc.k) + kv_block_offset<D, kInt4>(kc, page, h, slot >> 4);
  uint4 w;
  if (kInt4) {
    uint32_t codes, x[4];
    float s;
    load4<D>(block, slot & 15, c, value, codes, s);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float a = (float)((int)((codes >> (8 * n)) & 15u) - 8) * s;
      const float d = (float)((int)((codes >> (8 * n + 4)) & 15u) - 8) * s;
      x[n] = pack_bf16x2(a, d);
    }
    w = make_uint4(x[0], x[1], x[2], x[3]);
  } else {
    w = *reinterpret_cast<const uint4*>(block + (slot & 15) * D * 2 + 16 * c);
  }
  uint16_t* out = value ? p.v_out : p.k_out;
  *reinterpret_cast<uint4*>(out + (((long long)b * kc.H_kv + h) * p.S + i) * D + 8 * c) = w;
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p0, int D, bool int4, cudaStream_t stream) {
  KvAppendParams p = p0;
  const int slots = kKvThreads / (D / 8);
  const int rows = p.H_q + 2 * p.cache.H_kv;
  p.rounds = 1;
  const int ny = (rows + slots * p.rounds - 1) / (slots * p.rounds);
  const dim3 grid((unsigned)((long long)p.cache.B * p.S), (unsigned)ny);
  if (D == 128 && int4) kv_append_kernel<128, true><<<grid, kKvThreads, 0, stream>>>(p);
  else if (D == 128) kv_append_kernel<128, false><<<grid, kKvThreads, 0, stream>>>(p);
  else if (int4) kv_append_kernel<64, true><<<grid, kKvThreads, 0, stream>>>(p);
  else kv_append_kernel<64, false><<<grid, kKvThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvReadParams& p, int D, bool int4, cudaStream_t stream) {
  const int slots = kKvThreads / (D / 8);
  const long long rows = (long long)p.cache.B * p.S;
  const dim3 grid((unsigned)((rows + slots - 1) / slots), (unsigned)(2 * p.cache.H_kv));
  if (D == 128 && int4) kv_read_kernel<128, true><<<grid, kKvThreads, 0, stream>>>(p);
  else if (D == 128) kv_read_kernel<128, false><<<grid, kKvThreads, 0, stream>>>(p);
  else if (int4) kv_read_kernel<64, true><<<grid, kKvThreads, 0, stream>>>(p);
  else kv_read_kernel<64, false><<<grid, kKvThreads, 0, stream>>>(p);
  return cudaGetLastError();
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
