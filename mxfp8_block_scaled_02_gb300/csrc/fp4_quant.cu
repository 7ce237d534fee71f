// fp4_quant.cu - bf16 -> MXFP4 / NVFP4, and packed E2M1 codes -> E4M3 bytes.
//
// Quantise (the rules are in mx_fp4.cuh): one lane per 32 consecutive elements
// (one MXFP4 block or two NVFP4 blocks), so no cross-lane step; a warp reads
// 2 KB and writes 512 bytes of codes.  Bound by HBM: 2 bytes read and 0.53
// (0.56) written per element.
//
// Unpack: an E2M1 value is an E4M3 value, so the codes widen exactly to one
// E4M3 byte each (an MXFP4 tensor becomes an MXFP8 one with the same E8M0
// scales).  A lane takes 16 bytes of codes and looks its nibbles up four at a
// time with a byte permute.  Bound by HBM: 0.5 bytes read, 1 written.
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_fp4.cuh"
#include "mx_kernels.h"
#include "mx_layout.cuh"
#include "mx_ptx.cuh"

namespace mx {

namespace {

constexpr int kThreads = 256;
constexpr int kU = 2;  // warp tasks per iteration, their loads all in flight

struct QuantArgs {
  const uint4* x;
  uint8_t* q;
  uint8_t* s;
  const float* g;  // NVFP4 tensor scale, or nullptr for 1
  uint32_t tasks;  // rows * K / 32
  uint32_t K32;    // K / 32
  uint32_t rows_per_b;
  uint32_t RT, KT;  // atom tiles of one batch (packed scales)
};

// kPacked: scales into the packed atoms, where the lane of a row's last task
// also zeroes the bytes that pad the row to whole words (a product that reads
// a whole word multiplies them with codes that are zero).  kEarly: as in
// quantize.cu, the activation quantise inside a linear call only.
template <int FMT, bool kPacked, bool kEarly>
__global__ void __launch_bounds__(kThreads) quantize_fp4_kernel(const QuantArgs a) {
  if (kEarly) {
    launch_dependents();
    grid_dependency_wait();
  }
  const float g = FMT == kQNV4 && a.g != nullptr ? __ldg(a.g) : 1.f;
  const float six_g = 6.f * g;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const uint32_t nwarps = (gridDim.x * blockDim.x) >> 5;
  const uint32_t ntasks = (a.tasks + 31) / 32;
  const int64_t atom_k_stride = static_cast<int64_t>(a.RT) * kAtomBytes;

  for (uint32_t t0 = warp * kU; t0 < ntasks; t0 += nwarps * kU) {
    uint4 v[kU][4];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t i = (t0 + u) * 32 + lane;
      const bool valid = t0 + u < ntasks && i < a.tasks;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[u][k] = valid ? __ldg(a.x + static_cast<uint64_t>(i) * 4 + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t i0 = (t0 + u) * 32;
      const uint32_t i = i0 + lane;
      if (t0 + u >= ntasks || i >= a.tasks) continue;
      uint4 codes;
      const uint32_t sb = quantize_fp4_32<FMT>(v[u], six_g, g, codes);
      reinterpret_cast<uint4*>(a.q)[i] = codes;
      if (!kPacked) {
        if (FMT == kQNV4)
          reinterpret_cast<uint16_t*>(a.s)[i] = static_cast<uint16_t>(sb);
        else
          a.s[i] = static_cast<uint8_t>(sb);
      } else {
        uint32_t row = i0 / a.K32;
        uint32_t k32 = i0 - row * a.K32 + lane;
        while (k32 >= a.K32) {
          k32 -= a.K32;
          ++row;
        }
        const uint32_t b = row / a.rows_per_b, r = row - b * a.rows_per_b;
        const uint32_t kb = FMT == kQNV4 ? 2 * k32 : k32;
        uint8_t* word = a.s + (static_cast<int64_t>(b) * a.KT * a.RT + (r >> 7)) * kAtomBytes + (r & 31) * 16 +
                        ((r >> 5) & 3) * 4 + (kb >> 2) * atom_k_stride;
        const uint32_t j = kb & 3;
        if (FMT == kQNV4) {
          *reinterpret_cast<uint16_t*>(word + j) = static_cast<uint16_t>(sb);
          if (k32 + 1 == a.K32 && j == 0) *reinterpret_cast<uint16_t*>(word + 2) = 0;
        } else {
          word[j] = static_cast<uint8_t>(sb);
          if (k32 + 1 == a.K32)
            for (uint32_t p = j + 1; p < 4; ++p) word[p] = 0;
        }
      }
    }
  }
}

// Four E2M1 codes (the low 16 bits of w) -> four E4M3 bytes.
__device__ __forceinline__ uint32_t e2m1x4_to_e4m3(uint32_t w) {
  const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, w & 0x7777u);
  const uint32_t sign = ((w & 0x8u) << 4) | ((w & 0x80u) << 8) | ((w & 0x800u) << 12) | ((w & 0x8000u) << 16);
  return mag | sign;
}

__global__ void __launch_bounds__(kThreads) fp4_unpack_kernel(const uint4* __restrict__ q, uint4* __restrict__ out,
                                                              uint64_t n) {
  const uint64_t stride = static_cast<uint64_t>(gridDim.x) * blockDim.x;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride) {
    const uint4 v = __ldg(q + i);
    out[2 * i] = make_uint4(e2m1x4_to_e4m3(v.x), e2m1x4_to_e4m3(v.x >> 16), e2m1x4_to_e4m3(v.y),
                            e2m1x4_to_e4m3(v.y >> 16));
    out[2 * i + 1] = make_uint4(e2m1x4_to_e4m3(v.z), e2m1x4_to_e4m3(v.z >> 16), e2m1x4_to_e4m3(v.w),
                                e2m1x4_to_e4m3(v.w >> 16));
  }
}

template <int FMT, bool kPacked, bool kEarly>
cudaError_t launch_t(const QuantArgs& a, int sms, cudaStream_t stream) {
  static int per_sm = 0;
  if (per_sm == 0) {
    int n = 0;
    cudaError_t e =
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, quantize_fp4_kernel<FMT, kPacked, kEarly>, kThreads, 0);
    per_sm = e == cudaSuccess && n > 0 ? n : 1;
  }
  const int64_t want = ceil_div(ceil_div(a.tasks, 32 * kU), kThreads / 32);
  const int64_t cap = static_cast<int64_t>(sms) * per_sm;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(want < cap ? want : cap), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kEarly ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, quantize_fp4_kernel<FMT, kPacked, kEarly>, a);
}

template <int FMT>
cudaError_t launch_fmt(const QuantArgs& a, bool packed, bool early, int sms, cudaStream_t stream) {
  if (packed) return early ? launch_t<FMT, true, true>(a, sms, stream) : launch_t<FMT, true, false>(a, sms, stream);
  return early ? launch_t<FMT, false, true>(a, sms, stream) : launch_t<FMT, false, false>(a, sms, stream);
}

}  // namespace

cudaError_t launch_quantize_fp4(int fmt, const void* x, int64_t B, int64_t M, int64_t K, const float* g, uint8_t* q,
                                uint8_t* s, bool packed_scales, int sms, cudaStream_t stream, bool early_trigger) {
  const int64_t tasks = B * M * (K / 32);
  if (tasks == 0) return cudaSuccess;
  if (tasks > kMaxBlocks32) return cudaErrorInvalidValue;  // the host refuses these first
  QuantArgs a;
  a.x = static_cast<const uint4*>(x);
  a.q = q;
  a.s = s;
  a.g = g;
  a.tasks = static_cast<uint32_t>(tasks);
  a.K32 = static_cast<uint32_t>(K / 32);
  a.rows_per_b = static_cast<uint32_t>(M);
  a.RT = static_cast<uint32_t>(ceil_div(M, kAtomRows));
  a.KT = static_cast<uint32_t>(ceil_div(fp4_scale_extent(fmt, K), kTileK));
  return fmt == kQNV4 ? launch_fmt<kQNV4>(a, packed_scales, early_trigger, sms, stream)
                      : launch_fmt<kQMX4>(a, packed_scales, early_trigger, sms, stream);
}

cudaError_t launch_fp4_unpack(const uint8_t* q, int64_t n, uint8_t* out, int sms, cudaStream_t stream) {
  const int64_t chunks = n / 32;
  if (chunks == 0) return cudaSuccess;
  const int64_t want = ceil_div(chunks, kThreads), cap = static_cast<int64_t>(sms) * 8;
  fp4_unpack_kernel<<<static_cast<unsigned>(want < cap ? want : cap), kThreads, 0, stream>>>(
      reinterpret_cast<const uint4*>(q), reinterpret_cast<uint4*>(out), static_cast<uint64_t>(chunks));
  return cudaGetLastError();
}

}  // namespace mx
