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
//     s = E4M3(amax / (6 g)) saturating at 448 (6 g at least 2^-149, the least
//     fp32, for the g = 0 of an all-zero tensor), element = E2M1(x * (1 / (s g)));
//     a zero block has s = 0, one whose s (or s g) is zero gets zero codes, one
//     holding Inf/NaN gets the scale 0x7F (NaN) and zero codes.  Every step is
//     one fp32 operation, rounded to nearest; any g >= 0 will do.
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

// E4M3 byte (finite, non-negative) -> fp32: its fields moved to fp32's, then the
// exponent rebiased by 2^(127 - 7), exactly (subnormals too).
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) { return __uint_as_float(b << 20) * 1.329227996e36f; }

// max(|a|, |b|), NaN if either is.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// NVFP4's tensor scale g and what the blocks share of it.
struct TensorScale {
  float g, six_g, inv_lo, inv_hi;
};

__device__ __forceinline__ TensorScale tensor_scale(float g) {
  // at least the least positive fp32: a zero block's 0 / (6 g) is 0 for g = 0 too
  // (a check beside the division took the activation 4096 x 14336 from 44.1 to 45.8 us)
  const float six_g = fmaxf(6.f * g, __uint_as_float(1u));
  // For 6 g in [2^-126, 2^126], where the quick division is good to 2 ulp: an
  // interval around 1 / (6 g), wider than those and a product's rounding.  Else
  // (its result may be 0, infinite or subnormal) ends that never round to the
  // same code, so that every block takes the exact division.
  const bool normal = six_g >= 1.17549435e-38f && six_g <= 8.50705917e37f;
  const float inv = __fdividef(1.f, six_g);
  return TensorScale{g, six_g, normal ? inv * (1.f - 9.53674316e-7f) : 0.f,
                     normal ? inv * (1.f + 9.53674316e-7f) : __uint_as_float(0x7F800000u)};
}

// A block's scale byte and the factor its elements are multiplied by, from the
// block's amax as a bit pattern of |x| in fp32 (integer order is value order;
// >= 0x7F800000 is Inf or NaN).
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, const TensorScale& ts, float* mul,
                                                bool* nonfinite) {
  *nonfinite = amax_bits >= 0x7F800000u;
  if (FMT == kQNV4) {
    // E4M3(amax / (6 g)) without the division, wherever both ends of the
    // interval around the quotient round to the same code
    const float amax = __uint_as_float(amax_bits);
    const uint32_t both = cvt_e4m3x2(amax * ts.inv_lo, amax * ts.inv_hi);
    uint32_t sb = both & 0xFFu;
    if (sb != both >> 8) sb = cvt_e4m3x2(__fdiv_rn(amax, ts.six_g), 0.f) & 0xFFu;
    const float g = ts.g;
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

// Quantise sixteen fp32 values per lane: a 16-element block is one lane, a
// 32-element block two neighbouring ones.  Every lane of the warp takes part.
// codes: 16 bytes of E4M3, or 8 bytes of E2M1 in codes[0..1].  Returns the
// block's scale byte (the same in its lanes).
template <int FMT>
__device__ __forceinline__ uint32_t quantize_lane16(const float (&v)[16], const TensorScale& ts, uint32_t (&codes)[4]) {
  float m4[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m4[i] = max_abs(max_abs(v[4 * i], v[4 * i + 1]), max_abs(v[4 * i + 2], v[4 * i + 3]));
  uint32_t m = __float_as_uint(max_abs(max_abs(m4[0], m4[1]), max_abs(m4[2], m4[3]))) & 0x7FFFFFFFu;
  if (FMT != kQNV4) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  float mul;
  bool nonfinite;
  const uint32_t sb = block_scale<FMT>(m, ts, &mul, &nonfinite);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[8 * h + i] * mul;
    if (FMT == kQMX8) {
      codes[2 * h] = cvt_e4m3x2(t[0], t[1]) | (cvt_e4m3x2(t[2], t[3]) << 16);
      codes[2 * h + 1] = cvt_e4m3x2(t[4], t[5]) | (cvt_e4m3x2(t[6], t[7]) << 16);
    } else {
      codes[h] = cvt_e2m1x8(t);
    }
  }
  if (nonfinite) {
#pragma unroll
    for (int i = 0; i < (FMT == kQMX8 ? 4 : 2); ++i) codes[i] = FMT == kQMX8 ? 0x7F7F7F7Fu : 0u;
  }
  return sb;
}

}  // namespace mx
