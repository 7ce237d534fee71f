// mx_fp4.cuh - 4-bit block quantisation (E2M1 elements) and the shared
// quantisation step of the fused norm and activation kernels.
//
// Two formats, both with E2M1 elements (0, .5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) packed two to a byte, the even element in the low half:
//   * MXFP4 (OCP MX v1.0, sections 5.3.3 and 6.3): one E8M0 scale per 32
//     elements, e = floor(log2 amax) - 2 clamped to [-127, 127], element =
//     E2M1(x / 2^e); a block holding Inf/NaN gets scale byte 0xFF and zero
//     codes (E2M1 has no NaN);
//   * NVFP4: one E4M3 scale per 16 elements and one fp32 scale g per tensor:
//     s = E4M3(amax / (6 g)) saturating at 448, element = E2M1(x * (1 / (s g)));
//     a block whose s (or s g) is zero gets zero codes, one holding Inf/NaN
//     gets the scale 0x7F (NaN) and zero codes.  Every step is one fp32
//     operation, rounded to nearest.
// Elements round to nearest even and saturate to +-6 (cvt.rn.satfinite).
//
// The scales' packed layout is the 512-byte atom of mx_layout.cuh (128 rows x
// 4 blocks): an atom covers 128 elements of K for MXFP4 and 64 for NVFP4, so
// every size and offset function there takes the "scale extent"
// fp4_scale_extent(fmt, K): K counted as if its blocks were 32 long.
#pragma once

#include <stdint.h>

#include "mx_layout.cuh"
#include "mx_ptx.cuh"

namespace mx {

// Output formats of the quantising kernels (MXFP8_QFMT_*).
constexpr int kQMX8 = 0;  // MXFP8: E4M3 elements, E8M0 scale per 32
constexpr int kQMX4 = 1;  // MXFP4
constexpr int kQNV4 = 2;  // NVFP4

__host__ __device__ constexpr int q_block(int fmt) { return fmt == kQNV4 ? 16 : 32; }
__host__ __device__ constexpr int64_t fp4_scale_extent(int fmt, int64_t K) { return fmt == kQNV4 ? 2 * K : K; }

// Eight fp32 -> eight E2M1 codes, element i in bits [4i, 4i + 4).
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// E4M3 byte (finite, non-negative) -> fp32, by its fields: exact.
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  const uint32_t e = b >> 3, m = b & 7u;
  return e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : static_cast<float>(m) * 0.001953125f;  // 2^-9
}

// A block's scale byte and the factor its elements are multiplied by, from the
// block's amax as a bit pattern of |x| in fp32 (integer order is value order;
// >= 0x7F800000 is Inf or NaN).  six_g and g are NVFP4's tensor scale.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, float six_g, float g, float* mul, bool* nonfinite) {
  *nonfinite = amax_bits >= 0x7F800000u;
  if (FMT == kQNV4) {
    const uint32_t sb = cvt_e4m3x2(__fdiv_rn(__uint_as_float(amax_bits), six_g), 0.f) & 0xFFu;
    const float unit = e4m3_to_f32(sb & 0x7Fu) * g;
    const float inv = __frcp_rn(unit);
    // a zero (or NaN) unit, or one so small that its inverse overflows: zero codes
    *mul = unit > 0.f && inv < __uint_as_float(0x7F800000u) ? inv : 0.f;
    return *nonfinite ? 0x7Fu : sb;
  }
  constexpr uint32_t kEmax = FMT == kQMX8 ? 8u : 2u;
  const uint32_t E = amax_bits >> 23;
  const uint32_t sb = *nonfinite ? 0xFFu : (E > kEmax ? E - kEmax : 0u);
  *mul = __uint_as_float((254u - (*nonfinite ? 0u : sb)) << 23);
  return sb;
}

// Quantise eight fp32 values per lane; a block is 4 (16-element NVFP4: 2)
// consecutive lanes.  Every lane of the warp takes part.  codes: 8 bytes of
// E4M3, or 4 bytes of E2M1 in codes.x.  Returns the block's scale byte (the
// same in its lanes).
template <int FMT>
__device__ __forceinline__ uint32_t quantize_lane8(const float (&v)[8], float six_g, float g, uint2& codes) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  if (FMT != kQNV4) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  float mul;
  bool nonfinite;
  const uint32_t sb = block_scale<FMT>(m, six_g, g, &mul, &nonfinite);
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = v[i] * mul;
  if (FMT == kQMX8) {
    codes.x = cvt_e4m3x2(t[0], t[1]) | (cvt_e4m3x2(t[2], t[3]) << 16);
    codes.y = cvt_e4m3x2(t[4], t[5]) | (cvt_e4m3x2(t[6], t[7]) << 16);
    if (nonfinite) codes.x = codes.y = 0x7F7F7F7Fu;
  } else {
    codes.x = nonfinite ? 0u : cvt_e2m1x8(t);
    codes.y = 0u;
  }
  return sb;
}

// 32 consecutive bf16 values in one lane (16 words) -> 16 bytes of E2M1 codes.
// The scale byte(s): MXFP4 one in bits [0, 8), NVFP4 two (the second block of
// 16 in bits [8, 16)).
template <int FMT>
__device__ __forceinline__ uint32_t quantize_fp4_32(const uint4 (&v)[4], float six_g, float g, uint4& codes) {
  uint32_t w[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    w[4 * q] = v[q].x;
    w[4 * q + 1] = v[q].y;
    w[4 * q + 2] = v[q].z;
    w[4 * q + 3] = v[q].w;
  }
  uint32_t m[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = __vmaxu2(a, w[8 * h + i] & 0x7FFF7FFFu);
    m[h] = max(a & 0xFFFFu, a >> 16) << 16;  // the bf16 amax as fp32 bits
  }
  float mul[2];
  bool bad[2];
  uint32_t sb;
  if (FMT == kQNV4) {
    sb = block_scale<FMT>(m[0], six_g, g, &mul[0], &bad[0]);
    sb |= block_scale<FMT>(m[1], six_g, g, &mul[1], &bad[1]) << 8;
  } else {
    sb = block_scale<FMT>(max(m[0], m[1]), six_g, g, &mul[0], &bad[0]);
    mul[1] = mul[0];
    bad[1] = bad[0];
  }
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[2 * i] = __uint_as_float(w[4 * q + i] << 16) * mul[q >> 1];
      t[2 * i + 1] = __uint_as_float(w[4 * q + i] & 0xFFFF0000u) * mul[q >> 1];
    }
    o[q] = bad[q >> 1] ? 0u : cvt_e2m1x8(t);
  }
  codes = make_uint4(o[0], o[1], o[2], o[3]);
  return sb;
}

}  // namespace mx
