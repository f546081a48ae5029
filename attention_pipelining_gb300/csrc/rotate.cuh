// rotate.cuh -- rotation of pairs of bf16 elements by (cos, sin), rounded once to bf16 from the
// exact value: shared by the cache's append kernel and the rotation of packed sequences.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace attnpipe {

// u a + w b of two pairs, rounded once to bf16 (returned as floats).  u and w are bf16
// values and a and b fp32, so the exact value may have more bits than a float:
// the products' and the sum's rounding errors are recovered (fma, two-sum) and
// added back, and the fp32 result, when it falls on a tie of the bf16 rounding
// that the remainder breaks, is moved one step to the remainder's side.  Non-finite
// values take the plain formula's result.  (A product's error has its 32 bits' last, 2^-30 of
// the product's factors' powers of two, and is a float where the product is 2^-117 or more; below
// that the errors are rounded to 2^-149, by 2^-150 each.)
__device__ __forceinline__ void rotate2_exactly(uint64_t u, uint64_t a, uint64_t w, uint64_t b,
                                                float& r0, float& r1) {
  const uint64_t minus = f2_pack(-1.f, -1.f);
  const auto sub = [&](uint64_t x, uint64_t y) { return f2_fma(y, minus, x); };
  const uint64_t h = f2_mul(u, a), h2 = f2_mul(w, b);
  const uint64_t e = f2_fma(u, a, f2_mul(h, minus)), e2 = f2_fma(w, b, f2_mul(h2, minus));
  const uint64_t s = f2_add(h, h2), t = sub(s, h);
  const uint64_t es = f2_add(sub(h, sub(s, t)), sub(h2, t));
  const uint64_t lo = f2_add(es, f2_add(e, e2)), r = f2_add(s, lo), rem = sub(lo, sub(r, s));
  float rr[2], ss[2], mm[2];
  f2_unpack(r, rr[0], rr[1]);
  f2_unpack(s, ss[0], ss[1]);
  f2_unpack(rem, mm[0], mm[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t x = __float_as_uint(rr[i]);
    if ((x & 0xffffu) == 0x8000u && mm[i] != 0.f)
      x += ((mm[i] > 0.f) == (rr[i] > 0.f)) ? 1u : 0xffffffffu;
    // an infinity or a NaN: the plain formula's
    rr[i] = fabsf(rr[i]) <= 3.4028235e38f ? __uint_as_float(x) : ss[i];
  }
  r0 = rr[0], r1 = rr[1];
}

// Four pairs: (x c - y s, y c + x s), first with five operations a result,
// fma(x, c, h) + e with h + e = -y s exactly, which is off by at most two units of
// fp32's last place (half a unit in each of the two sums, of which the first may
// be twice as large as the second's; the sum of products that cancel is exact);
// only where that leaves the bf16 rounding open (two units around a tie: one
// element in 13000) or a value is not finite, by rotate2_exactly.
// Rounding the plain fp32 formula instead would round about one element in 2^15
// the other way than the exact value, and in a 4-bit cache change its code.
__device__ __forceinline__ void rotate4(const uint64_t (&x)[2], const uint64_t (&y)[2],
                                        const uint64_t (&c)[2], const uint64_t (&s)[2],
                                        float (&r1)[4], float (&r2)[4]) {
  const uint64_t minus = f2_pack(-1.f, -1.f), zero = f2_pack(0.f, 0.f);
  uint32_t nearest = 0xffffffffu;   // of the first of each two, of the second
  uint64_t finite = zero;
  const auto one = [&](uint64_t u, uint64_t w, uint64_t cs, uint64_t sn, uint64_t minus_sn,
                       float& f0, float& f1) {   // u cs + w sn
    const uint64_t e = f2_fma(w, sn, f2_mul(w, minus_sn));
    const uint64_t r = f2_add(f2_fma(u, cs, f2_mul(w, sn)), e);
    finite = f2_fma(r, zero, finite);
    f2_unpack(r, f0, f1);
    nearest = __viaddmin_u16x2(
        __byte_perm(__float_as_uint(f0), __float_as_uint(f1), 0x5410u), 0x80028002u, nearest);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t ms = f2_mul(s[i], minus);
    one(x[i], y[i], c[i], ms, s[i], r1[2 * i], r1[2 * i + 1]);
    one(y[i], x[i], c[i], s[i], ms, r2[2 * i], r2[2 * i + 1]);
  }
  float f0, f1;
  f2_unpack(finite, f0, f1);
  if ((nearest & 0xffffu) <= 4u || (nearest >> 16) <= 4u || f0 + f1 != 0.f) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t ms = f2_mul(s[i], minus);
      rotate2_exactly(x[i], c[i], y[i], ms, r1[2 * i], r1[2 * i + 1]);
      rotate2_exactly(y[i], c[i], x[i], s[i], r2[2 * i], r2[2 * i + 1]);
    }
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The rotation of a lane's eight elements, w.x, w.y and w.z, w.w: four first
// and four second elements of its pairs, or (interleaved) four adjacent pairs.
template <bool kInterleaved>
__device__ __forceinline__ void rotate_lane(uint4& w, const uint64_t (&cs)[2],
                                            const uint64_t (&sn)[2]) {
  uint64_t x[2], y[2];
  float r1[4], r2[4];
  if constexpr (kInterleaved) {
    x[0] = f2_pack(bf16_lo(w.x), bf16_lo(w.y)), x[1] = f2_pack(bf16_lo(w.z), bf16_lo(w.w));
    y[0] = f2_pack(bf16_hi(w.x), bf16_hi(w.y)), y[1] = f2_pack(bf16_hi(w.z), bf16_hi(w.w));
  } else {
    x[0] = f2_pack(bf16_lo(w.x), bf16_hi(w.x)), x[1] = f2_pack(bf16_lo(w.y), bf16_hi(w.y));
    y[0] = f2_pack(bf16_lo(w.z), bf16_hi(w.z)), y[1] = f2_pack(bf16_lo(w.w), bf16_hi(w.w));
  }
  rotate4(x, y, cs, sn, r1, r2);
  w = kInterleaved ? make_uint4(pack_bf16x2(r1[0], r2[0]), pack_bf16x2(r1[1], r2[1]),
                                pack_bf16x2(r1[2], r2[2]), pack_bf16x2(r1[3], r2[3]))
                   : make_uint4(pack_bf16x2(r1[0], r1[1]), pack_bf16x2(r1[2], r1[3]),
                                pack_bf16x2(r2[0], r2[1]), pack_bf16x2(r2[2], r2[3]));
}

}  // namespace attnpipe
