// The row arithmetic of the appends: exact widening, the fp64 rotation of a row
// held by four lanes, and the 32-channel quantizer.
#pragma once

#include "common.cuh"

namespace kvq {

// 3-input fp32 max / min (sm_100)
template <bool MAX>
__device__ __forceinline__ float mm3(float a, float b, float c) {
  float r;
  if (MAX)
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  else
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// max / min of v0, v[1..31] as a depth-4 tree
template <bool MAX>
__device__ __forceinline__ float reduce32(float v0, const float (&v)[32]) {
  float a[11];
  a[0] = mm3<MAX>(v0, v[1], v[2]);
#pragma unroll
  for (int i = 1; i < 10; ++i) a[i] = mm3<MAX>(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
  a[10] = mm3<MAX>(v[30], v[31], v[31]);
  const float b0 = mm3<MAX>(a[0], a[1], a[2]), b1 = mm3<MAX>(a[3], a[4], a[5]);
  const float b2 = mm3<MAX>(a[6], a[7], a[8]), b3 = mm3<MAX>(a[9], a[10], a[10]);
  return mm3<MAX>(mm3<MAX>(b0, b1, b2), b3, b3);
}

// 1.5 * 2^23: for 0 <= q <= 2^22, q + kRoundMagic rounds q to the nearest
// integer (ties to even) and leaves it in the low significand bits
constexpr float kRoundMagic = 12582912.0f;
constexpr float kNear = 0.5f - 1e-5f;  // |q - round(q)| beyond this: next to a rounding boundary

// low bytes of four words -> one word, a in byte 0
__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// four codes (bytes 0..3 of x, each < 2^BITS) -> one BITS*4-bit word, byte 0 lowest
template <int BITS>
__device__ __forceinline__ uint32_t compress_codes(uint32_t x) {
  if (BITS == 4) {
    x |= x >> 4;  // byte 0: c0 | c1 << 4, byte 2: c2 | c3 << 4
    return __byte_perm(x, 0, 0x0020) & 0xFFFFu;
  } else {
    x |= x >> 6;  // byte 0: c0 | c1 << 2, byte 2: c2 | c3 << 2
    return (x | (x >> 12)) & 0xFFu;
  }
}

// Quantize one 32-channel group held by this lane (v[0..31]); skip0: element 0
// is kept out of the range and gets code 0; clip: the clipping ratio applied to
// the group's minimum and maximum.  Returns the fp16 (scale, zero) pair; byte j
// of packed[p] is the code of element 4p + j.
//
// The code is round_half_even((x - zero) / scale) clamped to [0, L], the
// quotient as IEEE fp32 division gives it.  It is formed as
// q = (x - zero) * rcp(scale) with a correctly rounded reciprocal and clamped
// to [0, L] (the bounds are integers, so clamp and round commute); q is then
// within 2^-22 * q < 4e-6 of the clamped IEEE quotient.  When an element's q
// lies within 1e-5 of a rounding boundary (k + 1/2) the group is coded again
// with the IEEE division for such elements, so every code is the division's.
template <int BITS>
__device__ __forceinline__ __half2 quantize_group32(const float (&v)[32], bool skip0, float clip,
                                                   uint32_t (&packed)[8]) {
  const float v0 = skip0 ? v[1] : v[0];
  // -0 and +0 are the same extreme; take it as +0 so the stored bits are unique;
  // then the clipping ratio scales both ends (exact for clip = 1)
  const float mn = __fmul_rn(clip, __fadd_rn(reduce32<false>(v0, v), 0.0f));
  const float mx = __fmul_rn(clip, __fadd_rn(reduce32<true>(v0, v), 0.0f));
  constexpr int L = (1 << BITS) - 1;
  const float s32 = fminf(__fdiv_rn(__fsub_rn(mx, mn), (float)L), 65504.0f);
  const float zc = fminf(fmaxf(mn, -65504.0f), 65504.0f);
  const __half s16 = __float2half_rn(s32), z16 = __float2half_rn(zc);
  const float sf = __half2float(s16), zf = __half2float(z16);
  const float rs = sf != 0.0f ? __frcp_rn(sf) : 0.0f;  // sf == 0: every code is 0
  float near[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    uint32_t m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(v[4 * p + j], zf), rs), 0.0f), (float)L);
      const float mq = __fadd_rn(q, kRoundMagic);
      const float d = fabsf(__fsub_rn(q, __fsub_rn(mq, kRoundMagic)));  // exact: |q - round(q)|
      near[j] = fmaxf(near[j], (p == 0 && j == 0 && skip0) ? 0.0f : d);
      m[j] = __float_as_uint(mq);
    }
    packed[p] = pack_low_bytes(m[0], m[1], m[2], m[3]);
  }
  if (mm3<true>(mm3<true>(near[0], near[1], near[2]), near[3], near[3]) > kNear) {
    // rare: code the group again, with the IEEE division next to a boundary
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t m[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float d = __fsub_rn(v[4 * p + j], zf);
        float q = fminf(fmaxf(__fmul_rn(d, rs), 0.0f), (float)L);
        if (fabsf(__fsub_rn(q, rintf(q))) > kNear) q = fminf(fmaxf(rintf(__fdiv_rn(d, sf)), 0.0f), (float)L);
        m[j] = __float_as_uint(__fadd_rn(q, kRoundMagic));
      }
      packed[p] = pack_low_bytes(m[0], m[1], m[2], m[3]);
    }
  }
  if (skip0) packed[0] &= 0xFFFFFF00u;
  return __halves2half2(s16, z16);
}

// The same quantizer, bit for bit, in fewer instructions (about 5 per element instead of
// 8), for the paged append.
//
// Codes: the IEEE division's, as above.  t = sat(v c1 + c0) with c1 = 1 / (s L),
// c0 = -z c1 is q / L clamped; 128 + 1/2 + L t then holds q + 1/2 with 16 fraction
// bits in its significand, and byte 2 is q rounded.  With u = 2^-24 and
// |z| / s <= 30: |v c1| 3u + |z c1| 4u + |t| u of t is at most 270 u in q (1.05 units
// of 2^-16), the last rounding half a unit, the division's own error 30 u; so a
// q more than 2 units from a boundary rounds as the division's quotient.  Groups with
// an element nearer than that (6e-5 of the elements), or farther from zero than 30
// scales, are coded again with the IEEE division.
template <int BITS>
__device__ __forceinline__ __half2 quantize_group32_fast(float (&v)[32], bool skip0, float clip, uint32_t (&packed)[8]) {
  const float own0 = v[0];
  if (skip0) v[0] = v[1];
  const float mn = __fmul_rn(clip, __fadd_rn(reduce32<false>(v[0], v), 0.0f));
  const float mx = __fmul_rn(clip, __fadd_rn(reduce32<true>(v[0], v), 0.0f));
  constexpr int L = (1 << BITS) - 1;
  const float s32 = fminf(__fdiv_rn(__fsub_rn(mx, mn), (float)L), 65504.0f);
  const __half s16 = __float2half_rn(s32), z16 = __float2half_rn(fminf(fmaxf(mn, -65504.0f), 65504.0f));
  const float sf = __half2float(s16), zf = __half2float(z16);
  const float rs = sf != 0.0f ? __frcp_rn(sf) : 0.0f;  // sf == 0: every code is 0
  const float c1 = __fmul_rn(rs, 1.0f / L), c0 = -__fmul_rn(zf, c1);
  constexpr uint32_t kWindow = 2;
  constexpr float kMagic = 128.5f + kWindow / 65536.0f;
  uint32_t near = 0xFFFFFFFFu;  // least distance from a boundary, two elements side by side
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    uint32_t m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float t;
      asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(t) : "f"(v[4 * p + j]), "f"(c1), "f"(c0));
      m[j] = __float_as_uint(__fmaf_rn(t, (float)L, kMagic));
    }
    near = __vminu2(near, __vminu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[2], m[3], 0x5410)));
    packed[p] = __byte_perm(__byte_perm(m[0], m[1], 0x0062), __byte_perm(m[2], m[3], 0x0062), 0x5410);
  }
  const bool far = fabsf(zf) * rs > 30.0f;
  if (min(near & 0xFFFFu, near >> 16) <= 2 * kWindow || far) {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      float t;
      asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(t) : "f"(v[e]), "f"(c1), "f"(c0));
      const uint32_t m = __float_as_uint(__fmaf_rn(t, (float)L, kMagic));
      if ((m & 0xFFFFu) <= 2 * kWindow || far) {
        const float q = sf != 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[e], zf), sf)), 0.0f), (float)L) : 0.0f;
        const uint32_t code = (uint32_t)q;
        packed[e >> 2] = (packed[e >> 2] & ~(0xFFu << (8 * (e & 3)))) | (code << (8 * (e & 3)));
      }
    }
  }
  if (skip0) {
    packed[0] &= 0xFFFFFF00u;
    v[0] = own0;
  }
  return __halves2half2(s16, z16);
}

// 32 consecutive input elements held raw: 64 bytes (16-bit types) or 128 (fp32)
template <typename In>
struct Raw32 {
  uint4 w[sizeof(In) * 2];
};
template <typename In>
__device__ __forceinline__ void load_raw(const In* p, Raw32<In>& r) {
#pragma unroll
  for (int j = 0; j < (int)sizeof(In) * 2; ++j) r.w[j] = reinterpret_cast<const uint4*>(p)[j];
}
__device__ __forceinline__ void widen2(uint32_t u, const __nv_bfloat16*, float& a, float& b) {
  a = __uint_as_float(u << 16);
  b = __uint_as_float(u & 0xFFFF0000u);
}
__device__ __forceinline__ void widen2(uint32_t u, const __half*, float& a, float& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
  a = f.x;
  b = f.y;
}
// exact widening to fp32
template <typename In>
__device__ __forceinline__ void widen(const Raw32<In>& r, float (&f)[32]) {
  if constexpr (sizeof(In) == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[4 * j] = __uint_as_float(r.w[j].x);
      f[4 * j + 1] = __uint_as_float(r.w[j].y);
      f[4 * j + 2] = __uint_as_float(r.w[j].z);
      f[4 * j + 3] = __uint_as_float(r.w[j].w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      widen2(r.w[j].x, (const In*)nullptr, f[8 * j], f[8 * j + 1]);
      widen2(r.w[j].y, (const In*)nullptr, f[8 * j + 2], f[8 * j + 3]);
      widen2(r.w[j].z, (const In*)nullptr, f[8 * j + 4], f[8 * j + 5]);
      widen2(r.w[j].w, (const In*)nullptr, f[8 * j + 6], f[8 * j + 7]);
    }
  }
}

// Orthonormal Walsh-Hadamard transform of one 128-channel row held by four
// lanes, lane g holding channels 32g .. 32g+31: butterflies in fp64, natural
// Sylvester order (stage h pairs channels i and i + h, i & h == 0, -> (a + b,
// a - b)); the stages below 32 stay inside the lane, 32 and 64 pair lanes g ^ 1
// and g ^ 2; then one fp64 multiply by 1/sqrt(128) and a round to fp32.  All
// 32 lanes of the warp take part.
__device__ __forceinline__ void rotate_row_4lanes(float (&v)[32], int g, double inv_sqrt_d) {
  double x[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = v[i];
#pragma unroll
  for (int hs = 1; hs < 32; hs <<= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if ((i & hs) == 0) {
        const double u = x[i], w = x[i + hs];
        x[i] = __dadd_rn(u, w);
        x[i + hs] = __dsub_rn(u, w);
      }
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    const bool upper = (g & m) != 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      // lower lane: x + o; upper lane: o - x = o + (-x), the same IEEE sum
      const double o = __shfl_xor_sync(kFull, x[i], m);
      x[i] = __dadd_rn(upper ? -x[i] : x[i], o);
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __double2float_rn(__dmul_rn(x[i], inv_sqrt_d));
}

}  // namespace kvq
