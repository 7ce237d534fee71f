// mx_block128.cuh - the fp8_128 quantisation step of the quantising kernels and of the
// few-token product.
//
// A block of 128 elements has the fp32 scale s = amax / 448 and the codes
// E4M3(448 x / amax), to nearest even, of the exact quotient: x and amax have 8
// significant bits, so 448 x / amax is either a tie of two codes, which has at
// most 5, or at least 1 / 7905 away from one (relative; 7905 = 31 * 255).  The fp32
// product x * (448 / amax) is off by at most 2 ulp, so rounded to 17 bits it is
// exactly the tie where there is one and on the right side elsewhere; no division
// per element is needed.  A zero block has s = 0 and zero codes (the signs kept), a
// block that holds Inf or NaN s = NaN and the codes 0x7F, as MXFP8's blocks.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "mx_ptx.cuh"

namespace mx {

// 448 / amax, and what x is multiplied by before it (a power of two: 1 but for an
// amax so small that the quotient would overflow).
__device__ __forceinline__ float b128_inverse(float amax, float* pre) {
  *pre = amax < 0x1p-110f ? 0x1p100f : 1.f;
  return amax > 0.f ? __fdiv_rn(448.f, amax * *pre) : 0.f;
}

// x * inv to 17 significant bits (see above); for values that are not of 16 bits
// this moves a quotient by 2^-17, an E4M3 tie's neighbourhood of 2^-13 of a step.
__device__ __forceinline__ float b128_quotient(float x, float inv) {
  return __uint_as_float((__float_as_uint(x * inv) + 0x40u) & 0xFFFFFF80u);
}

struct Codes {
  uint32_t w[4];
};

// Sixteen bf16 of a lane, eight lanes a block of 128 (absent elements are zero):
// the codes, and the block's scale in each of the eight lanes.
__device__ __forceinline__ Codes quantize16_b128(const uint32_t (&v)[8], float* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  const bool nonfinite = m >= 0x7F80u;
  const float amax = __uint_as_float(m << 16);
  float pre;
  const float inv = b128_inverse(amax, &pre);
  *scale = nonfinite ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 448.f);
  Codes c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f[2 * j] = __uint_as_float(v[2 * i + j] << 16);
      f[2 * j + 1] = __uint_as_float(v[2 * i + j] & 0xFFFF0000u);
    }
    if (pre != 1.f) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] *= pre;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = b128_quotient(f[j], inv);
    c.w[i] = nonfinite ? 0x7F7F7F7Fu : cvt_e4m3x2(f[0], f[1]) | (cvt_e4m3x2(f[2], f[3]) << 16);
  }
  return c;
}

// The same of fp32 values (an activation's): no quotient here is close to a tie by
// construction, and none is snapped to one.
__device__ __forceinline__ Codes quantize16_b128(const float (&y)[16], float* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  const bool nonfinite = m >= 0x7F800000u;
  const float amax = __uint_as_float(m);
  float pre;
  const float inv = b128_inverse(amax, &pre);
  *scale = nonfinite ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 448.f);
  Codes c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = cvt_e4m3x2(y[4 * i] * pre * inv, y[4 * i + 1] * pre * inv);
    const uint32_t b = cvt_e4m3x2(y[4 * i + 2] * pre * inv, y[4 * i + 3] * pre * inv);
    c.w[i] = nonfinite ? 0x7F7F7F7Fu : a | (b << 16);
  }
  return c;
}

// 16 bf16 at a 16-byte (wide: 32-byte) aligned address.
__device__ __forceinline__ void load16(const __nv_bfloat16* p, bool wide, uint32_t (&v)[8]) {
  if (wide) {
    ld_global_32(p, v);
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

}  // namespace mx
