// fused_quant.cu - the steps that feed a quantised linear layer, each with its
// output already quantised (MXFP8, MXFP4 or NVFP4; rules in mx_fp4.cuh):
//
//   rmsnorm : t = x + residual (fp32), y = t * rsqrt(mean(t^2) + eps) * w,
//             outputs quantise(y), t rounded once to the residual's type, and
//             optionally y as bf16;
//   silu_mul: y = gate / (1 + exp(-gate)) * up, output quantise(y).
//
// y stays in fp32 from the sum to the element's rounding: it is rounded once.
// Both read each input once and write each output once, and are bound by HBM
// on long inputs and by one round trip to memory on short ones.
//
// A thread owns chunks of 8 consecutive elements (one 16-byte load of bf16), so
// a 32-element block is 4 neighbouring lanes and its amax two shuffles; the
// codes of a warp's chunks are contiguous.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_fp4.cuh"
#include "mx_kernels.h"
#include "mx_layout.cuh"
#include "mx_ptx.cuh"

namespace mx {

namespace {

// Where a row's quantised chunks go.  RT == 0: row-major scales.
struct QuantOut {
  uint8_t* q;
  uint8_t* s;
  const float* g;  // NVFP4 tensor scale, or nullptr for 1
  int64_t K;       // elements per row
  int64_t RT;      // atom row tiles (packed scales)
};

__device__ __forceinline__ void unpack_bf16x8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Quantise chunk `c` (8 elements) of row `row` and store it.  Every lane of the
// warp calls; only valid lanes store.  A row is whole blocks, so the lanes of a
// block are valid together.
template <int FMT>
__device__ __forceinline__ void quantize_store(const QuantOut& o, int64_t row, int c, bool valid, const float (&y)[8],
                                               float six_g, float g) {
  uint2 codes;
  const uint32_t sb = quantize_lane8<FMT>(y, six_g, g, codes);
  if (!valid) return;
  constexpr int kLanes = q_block(FMT) / 8;
  if (FMT == kQMX8)
    *reinterpret_cast<uint2*>(o.q + row * o.K + 8 * static_cast<int64_t>(c)) = codes;
  else
    *reinterpret_cast<uint32_t*>(o.q + (row * o.K + 8 * static_cast<int64_t>(c)) / 2) = codes.x;
  if (c % kLanes != 0) return;
  const int64_t KB = o.K / q_block(FMT), kb = c / kLanes;
  if (o.RT == 0) {
    o.s[row * KB + kb] = static_cast<uint8_t>(sb);
    return;
  }
  uint8_t* word = o.s + ((kb >> 2) * o.RT + (row >> 7)) * kAtomBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
  word[kb & 3] = static_cast<uint8_t>(sb);
  if (kb + 1 == KB)  // the bytes that pad the row to whole scale words are zero
    for (int64_t p = (kb & 3) + 1; p < 4; ++p) word[p] = 0;
}

struct NormArgs {
  const __nv_bfloat16* x;
  int64_t x_stride;
  const void* res;  // bf16 or fp32 rows, or nullptr
  int64_t res_stride;
  void* res_out;    // dense rows of the residual's type
  const __nv_bfloat16* w;
  __nv_bfloat16* y;  // dense bf16 rows, or nullptr
  float eps;
  QuantOut o;
};

enum { kResNone = 0, kResBf16 = 1, kResF32 = 2 };

constexpr int norm_max_threads(int ch) { return ch == 1 ? 1024 : 512; }
// With few chunks a thread the weight is loaded up front (a short call's
// latency); with many, each SM has other rows to run while it is fetched from
// L2, and the registers are worth more.
template <int CH>
constexpr bool kPreloadW = CH <= 2;

// One CTA per row, the row held in registers (CH chunks a thread) between the
// sum of squares and the output, so x and the residual are read once.  The
// norm's weight and the tensor scale depend on nothing the kernel before this
// one writes and are read before the dependency wait; the next kernel in the
// stream may start at once (a GEMM that reads the output after its own wait).
template <int FMT, int CH, int RES>
__global__ void __launch_bounds__(norm_max_threads(CH)) rmsnorm_kernel(const NormArgs a) {
  __shared__ float part[32];
  launch_dependents();
  const int64_t row = blockIdx.x;
  const int nchunks = static_cast<int>(a.o.K / 8);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint4* wp = reinterpret_cast<const uint4*>(a.w);
  uint4 w[kPreloadW<CH> ? CH : 1];
  if (kPreloadW<CH>) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      w[i] = c < nchunks ? __ldg(wp + c) : make_uint4(0, 0, 0, 0);
    }
  }
  grid_dependency_wait();
  float t[CH][8];
  {
    uint4 xv[CH], r0[CH], r1[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      const uint4 z = make_uint4(0, 0, 0, 0);
      xv[i] = r0[i] = r1[i] = z;
      if (c >= nchunks) continue;
      xv[i] = *(reinterpret_cast<const uint4*>(a.x + row * a.x_stride) + c);
      if (RES == kResBf16)
        r0[i] = *(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.res) + row * a.res_stride) + c);
      if (RES == kResF32) {
        const uint4* rp = reinterpret_cast<const uint4*>(static_cast<const float*>(a.res) + row * a.res_stride) + 2 * c;
        r0[i] = rp[0];
        r1[i] = rp[1];
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      unpack_bf16x8(xv[i], t[i]);
      if (RES == kResBf16) {
        float r[8];
        unpack_bf16x8(r0[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[i][j] += r[j];
      }
      if (RES == kResF32) {
        const uint32_t r[8] = {r0[i].x, r0[i].y, r0[i].z, r0[i].w, r1[i].x, r1[i].y, r1[i].z, r1[i].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) t[i][j] += __uint_as_float(r[j]);
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(t[i][j], t[i][j], ss);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  // every warp adds the partials itself, in the same order
  ss = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
  const float rstd = rsqrtf(ss / static_cast<float>(a.o.K) + a.eps);
  const float g = FMT == kQNV4 && a.o.g != nullptr ? *a.o.g : 1.f;
  const float six_g = 6.f * g;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (i > 0 && (c & ~31) >= nchunks) break;  // the whole warp is past the row
    const bool valid = c < nchunks;
    if (RES == kResBf16 && valid)
      *(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.res_out) + row * a.o.K) + c) = pack_bf16x8(t[i]);
    if (RES == kResF32 && valid) {
      float4* rp = reinterpret_cast<float4*>(static_cast<float*>(a.res_out) + row * a.o.K) + 2 * c;
      rp[0] = make_float4(t[i][0], t[i][1], t[i][2], t[i][3]);
      rp[1] = make_float4(t[i][4], t[i][5], t[i][6], t[i][7]);
    }
    float wf[8], y[8];
    unpack_bf16x8(kPreloadW<CH> ? w[kPreloadW<CH> ? i : 0] : (valid ? __ldg(wp + c) : make_uint4(0, 0, 0, 0)), wf);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = t[i][j] * rstd * wf[j];
    if (a.y != nullptr && valid) *(reinterpret_cast<uint4*>(a.y + row * a.o.K) + c) = pack_bf16x8(y);
    quantize_store<FMT>(a.o, row, c, valid, y, six_g, g);
  }
}

struct ActArgs {
  const __nv_bfloat16* gate;
  const __nv_bfloat16* up;
  int64_t gate_stride, up_stride;
  int segs;  // CTAs per row
  QuantOut o;
};

constexpr int kActThreads = 128;

// kActThreads x CH chunks of one row per CTA.
template <int FMT, int CH>
__global__ void __launch_bounds__(kActThreads) silu_mul_kernel(const ActArgs a) {
  launch_dependents();
  const int64_t row = blockIdx.x / a.segs;
  const int c0 = static_cast<int>(blockIdx.x - row * a.segs) * (kActThreads * CH) + threadIdx.x;
  const int nchunks = static_cast<int>(a.o.K / 8);
  grid_dependency_wait();
  uint4 gv[CH], uv[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + i * kActThreads;
    gv[i] = uv[i] = make_uint4(0, 0, 0, 0);
    if (c >= nchunks) continue;
    gv[i] = *(reinterpret_cast<const uint4*>(a.gate + row * a.gate_stride) + c);
    uv[i] = *(reinterpret_cast<const uint4*>(a.up + row * a.up_stride) + c);
  }
  const float g = FMT == kQNV4 && a.o.g != nullptr ? *a.o.g : 1.f;
  const float six_g = 6.f * g;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + i * kActThreads;
    if ((c & ~31) >= nchunks) break;
    float gt[8], up[8], y[8];
    unpack_bf16x8(gv[i], gt);
    unpack_bf16x8(uv[i], up);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // gate / (1 + exp(-gate)) with the exponential's argument <= 0, so that
      // nothing overflows and very negative gates keep their value
      const float e = __expf(-fabsf(gt[j]));
      y[j] = gt[j] * __fdividef(gt[j] >= 0.f ? 1.f : e, 1.f + e) * up[j];
    }
    quantize_store<FMT>(a.o, row, c, c < nchunks, y, six_g, g);
  }
}

cudaError_t launch_pdl(void* kern, int64_t grid, int threads, void* args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* params[1] = {args};
  return cudaLaunchKernelExC(&cfg, kern, params);
}

template <int FMT, int CH>
void* norm_kernel(int res) {
  return res == kResNone ? reinterpret_cast<void*>(rmsnorm_kernel<FMT, CH, kResNone>)
                         : (res == kResBf16 ? reinterpret_cast<void*>(rmsnorm_kernel<FMT, CH, kResBf16>)
                                            : reinterpret_cast<void*>(rmsnorm_kernel<FMT, CH, kResF32>));
}

template <int FMT>
void* norm_kernel(int ch, int res) {
  return ch == 1 ? norm_kernel<FMT, 1>(res) : (ch == 2 ? norm_kernel<FMT, 2>(res) : (ch == 4 ? norm_kernel<FMT, 4>(res) : norm_kernel<FMT, 8>(res)));
}

}  // namespace

cudaError_t launch_rmsnorm_quantize(const NormProblem& p, int sms, cudaStream_t stream) {
  if (p.M == 0) return cudaSuccess;
  NormArgs a;
  a.x = static_cast<const __nv_bfloat16*>(p.x);
  a.x_stride = p.x_stride;
  a.res = p.res;
  a.res_stride = p.res_stride;
  a.res_out = p.res_out;
  a.w = static_cast<const __nv_bfloat16*>(p.w);
  a.y = static_cast<__nv_bfloat16*>(p.y);
  a.eps = p.eps;
  a.o = QuantOut{p.q, p.s, p.g, p.K, p.packed ? ceil_div(p.M, kAtomRows) : 0};
  const int res = p.res == nullptr ? kResNone : (p.res_f32 ? kResF32 : kResBf16);
  const int64_t chunks = p.K / 8;
  // One chunk a thread while that fits a CTA; with more rows than the GPU runs
  // at once, four, so that each SM has several rows' loads in flight.
  int ch = p.M >= 4 * sms ? 4 : 1;
  while (ceil_div(chunks, ch) > norm_max_threads(ch)) ch *= 2;
  if (ch > 8) return cudaErrorInvalidValue;  // the host refuses these first
  const int threads = static_cast<int>(ceil_div(ceil_div(chunks, ch), 32) * 32);
  void* k = p.fmt == kQMX8 ? norm_kernel<kQMX8>(ch, res)
                           : (p.fmt == kQMX4 ? norm_kernel<kQMX4>(ch, res) : norm_kernel<kQNV4>(ch, res));
  return launch_pdl(k, p.M, threads, &a, stream);
}

cudaError_t launch_silu_mul_quantize(const ActProblem& p, int sms, cudaStream_t stream) {
  if (p.M == 0) return cudaSuccess;
  ActArgs a;
  a.gate = static_cast<const __nv_bfloat16*>(p.gate);
  a.up = static_cast<const __nv_bfloat16*>(p.up);
  a.gate_stride = p.gate_stride;
  a.up_stride = p.up_stride;
  a.o = QuantOut{p.q, p.s, p.g, p.K, p.packed ? ceil_div(p.M, kAtomRows) : 0};
  const int64_t chunks = p.K / 8;
  // two chunks a thread once that still gives every SM work
  const bool two = p.M * ceil_div(chunks, 2 * kActThreads) >= 4 * static_cast<int64_t>(sms);
  a.segs = static_cast<int>(ceil_div(chunks, two ? 2 * kActThreads : kActThreads));
  const int64_t grid = p.M * a.segs;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;  // the host refuses these first
  void* k;
  if (two)
    k = p.fmt == kQMX8 ? reinterpret_cast<void*>(silu_mul_kernel<kQMX8, 2>)
                       : (p.fmt == kQMX4 ? reinterpret_cast<void*>(silu_mul_kernel<kQMX4, 2>)
                                         : reinterpret_cast<void*>(silu_mul_kernel<kQNV4, 2>));
  else
    k = p.fmt == kQMX8 ? reinterpret_cast<void*>(silu_mul_kernel<kQMX8, 1>)
                       : (p.fmt == kQMX4 ? reinterpret_cast<void*>(silu_mul_kernel<kQMX4, 1>)
                                         : reinterpret_cast<void*>(silu_mul_kernel<kQNV4, 1>));
  return launch_pdl(k, grid, kActThreads, &a, stream);
}

}  // namespace mx
