// Device building blocks of the 8-bit kernels: E4M3 conversion under a
// power-of-two scale (the rule is in include/averis.h), magnitudes, the scale
// bytes' layout, and the quantizer of a 512-column strip by one warp.
#pragma once

#include <cuda_bf16.h>

#include "device.cuh"

namespace avr {
namespace fp8 {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr uint32_t kInfBits = 0x7F800000u;

// scale byte e + 127 of a block whose largest magnitude has these bits: 448 =
// 1.75 * 2^8, so e = exponent - 8, one more when the significand passes 1.75
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const int b = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(b > 0 ? b : 0);
}
// 2^-e, exact: the byte is at most 247
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// two values -> two E4M3 codes, nearest even (lo in the low byte)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// four values times `inv` (a power of two: exact) -> four codes
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float inv) {
  float x0, x1, x2, x3;
  fmul2(a, b, inv, x0, x1);
  fmul2(c, d, inv, x2, x3);
  return __byte_perm(e4m3x2(x0, x1), e4m3x2(x2, x3), 0x5410);
}

// 16 bytes of input: kN values in 4 words
template <bool kBf16>
struct In {
  static constexpr int kN = kBf16 ? 8 : 4;
};
template <bool kBf16>
__device__ __forceinline__ float value_of(const uint4& q, int i) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (!kBf16) return __uint_as_float(w[i]);
  return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
}
// max(|a|, |b|) of words of two bf16 or one fp32; a NaN stays
template <bool kBf16>
__device__ __forceinline__ uint32_t abs_max(uint32_t a, uint32_t b) {
  if (kBf16) {
    const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(__uint_as_float(a))), "f"(fabsf(__uint_as_float(b))));
  return __float_as_uint(m);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t abs_max(const uint4& q) {
  return abs_max<kBf16>(abs_max<kBf16>(q.x, q.y), abs_max<kBf16>(q.z, q.w));
}
// the bits, as fp32's, of the larger value in a word that abs_max gave
template <bool kBf16>
__device__ __forceinline__ uint32_t amax_bits(uint32_t m) {
  return kBf16 ? max(m & 0xFFFF0000u, m << 16) : m;
}

// byte of (row r, block c) in the atom layout
__device__ __forceinline__ int64_t scale_at(int64_t r, int64_t c, int64_t atoms) {
  return ((r >> 7) * atoms + (c >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (c & 3);
}

// 512 columns of a row by a warp, 16 a lane (zeros past the row's end): the
// lane's codes, the four blocks' scale bytes as a word of an atom, and whether
// the block holds a NaN or an infinity
template <bool kBf16>
__device__ __forceinline__ void quant_strip(const uint4 (&q)[16 / In<kBf16>::kN], uint4* codes, uint32_t* word,
                                            bool* bad) {
  constexpr int N = In<kBf16>::kN, Q = 16 / N;
  uint32_t m = abs_max<kBf16>(q[0]);
#pragma unroll
  for (int i = 1; i < Q; ++i) m = abs_max<kBf16>(m, abs_max<kBf16>(q[i]));
  m = amax_bits<kBf16>(m);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
  *bad |= m >= kInfBits;
  const uint32_t byte = scale_byte(m);
  const float inv = inv_scale(byte);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) f[c] = value_of<kBf16>(q[(4 * i + c) / N], (4 * i + c) % N);
    w[i] = e4m3x4(f[0], f[1], f[2], f[3], inv);
  }
  *codes = make_uint4(w[0], w[1], w[2], w[3]);
  const int lane = threadIdx.x & 31;
  *word = __reduce_or_sync(kFull, (lane & 7) == 0 ? byte << (lane & 24) : 0u);
}

}  // namespace fp8
}  // namespace avr
