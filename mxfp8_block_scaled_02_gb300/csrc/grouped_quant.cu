// grouped_quant.cu - the quantising steps around the grouped and block-128 products:
// rows of x (in order, or picked by an index) and silu(gate) * up to E4M3 codes, and
// weights to codes with one scale per 128 x 128 block.
//
// fp8_128: the rule of mx_block128.cuh.
//
// MXFP8: the rule and the bytes of mx_quant.cuh.
//
// Bound by reading x and writing the codes.  Sixteen elements a lane (32 bytes in,
// 16 out: whole sectors), a block of 128 eight lanes, 512 elements a warp; one task a
// warp, many warps.  (Two or four tasks a warp with their loads first are slower: 4096
// x 14336 silu 52.4 us with one, 57.0 with two, both at six CTAs an SM; picked
// rows +1 % with two, +4 % with four.  16384 x 4096 quantised 39.2 us, 5.2 TB/s: the issue
// slots are 85 % busy, 38.8 with CTAs of 128 threads, 40.8 of 512, 39.1 with fewer
// instructions a division or an index.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_block128.cuh"
#include "mx_grouped.h"
#include "mx_layout.cuh"
#include "mx_ptx.cuh"
#include "mx_quant.cuh"

namespace mx {

namespace {

constexpr int THREADS = 256;
constexpr int TASK = 512;  // elements of a row per warp and task

// Sixteen bf16 of a lane, two lanes an MXFP8 block: the codes, and in the eight
// lanes of 128 elements the word of their four scale bytes.
__device__ __forceinline__ Codes quantize16_mx(const uint32_t (&v)[8], int lane, uint32_t* word) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  const bool nonfinite = m >= 0x7F80u;
  const uint32_t E = m >> 7;
  const uint32_t sbyte = nonfinite ? 0xFFu : (E > 8u ? E - 8u : 0u);
  const float mul = __uint_as_float((254u - (nonfinite ? 0u : sbyte)) << 23);
  uint32_t w = sbyte << (8 * ((lane >> 1) & 3));
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2);
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
  *word = w;
  Codes c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = cvt_e4m3x2(__uint_as_float(v[2 * i] << 16) * mul, __uint_as_float(v[2 * i] & 0xFFFF0000u) * mul);
    const uint32_t b =
        cvt_e4m3x2(__uint_as_float(v[2 * i + 1] << 16) * mul, __uint_as_float(v[2 * i + 1] & 0xFFFF0000u) * mul);
    c.w[i] = nonfinite ? 0x7F7F7F7Fu : a | (b << 16);
  }
  return c;
}

// The same of fp32 values, whose exponent decides as bf16's does.
__device__ __forceinline__ Codes quantize16_mx(const float (&y)[16], int lane, uint32_t* word) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  const bool nonfinite = m >= 0x7F800000u;
  const uint32_t E = m >> 23;
  const uint32_t sbyte = nonfinite ? 0xFFu : (E > 8u ? E - 8u : 0u);
  const float mul = __uint_as_float((254u - (nonfinite ? 0u : sbyte)) << 23);
  uint32_t w = sbyte << (8 * ((lane >> 1) & 3));
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2);
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
  *word = w;
  Codes c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = cvt_e4m3x2(y[4 * i] * mul, y[4 * i + 1] * mul);
    const uint32_t b = cvt_e4m3x2(y[4 * i + 2] * mul, y[4 * i + 3] * mul);
    c.w[i] = nonfinite ? 0x7F7F7F7Fu : a | (b << 16);
  }
  return c;
}

// Scale words [R][KT] -> [KT][R], 32 x 32 a CTA.
__global__ void __launch_bounds__(THREADS) transpose_words_kernel(const uint32_t* __restrict__ in, int64_t R, int KT,
                                                                  uint32_t* __restrict__ out) {
  __shared__ uint32_t box[32][33];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32;
  const int k0 = blockIdx.y * 32, x = threadIdx.x & 31, y = threadIdx.x >> 5;
  grid_dependency_wait();
  launch_dependents();  // in this order, as above
#pragma unroll
  for (int i = 0; i < 32; i += THREADS / 32)
    if (r0 + y + i < R && k0 + x < KT) box[y + i][x] = in[(r0 + y + i) * KT + k0 + x];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 32; i += THREADS / 32)
    if (r0 + x < R && k0 + y + i < KT) out[static_cast<int64_t>(k0 + y + i) * R + r0 + x] = box[x][y + i];
}

struct RowsArgs {
  const __nv_bfloat16* x;
  const int* rows;
  const int* positions;
  int k;          // positions a row of x
  int64_t T, R, K;
  int64_t tasks;  // (R, or T with positions) * segs
  int segs;       // tasks a row
  bool wide;
  uint8_t* q;
  uint32_t* s;
  int64_t s_row, s_kt;
};

// K % 16 == 0; MXFP8 K % 128 == 0.
template <int FMT, bool kEarly>
__global__ void __launch_bounds__(THREADS) quantize_rows_kernel(const RowsArgs a) {
  // In this order: when the next kernel starts, all before this one is done, and it
  // may read what this one does not write (GroupedProblem::offsets_ready).
  if (kEarly) {
    grid_dependency_wait();
    launch_dependents();
  }
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
  if (task >= a.tasks) return;  // the whole warp
  const int64_t row = task / a.segs;
  const int k = static_cast<int>(task - row * a.segs) * TASK + lane * 16;
  const int64_t src = a.rows != nullptr ? a.rows[row] : row;
  int pos = -1;  // lane j: where copy j of this row goes
  if (a.positions != nullptr && lane < a.k) pos = a.positions[row * a.k + lane];
  uint32_t v[8] = {};
  if (k < a.K && src >= 0 && src < a.T) load16(a.x + src * a.K + k, a.wide, v);
  uint32_t word;
  Codes c;
  if (FMT == kG8MX) {
    c = quantize16_mx(v, lane, &word);
  } else {
    float s;
    c = quantize16_b128(v, &s);
    word = __float_as_uint(s);
  }
  auto store = [&](int64_t r) {
    if (k < a.K) {
      *reinterpret_cast<uint4*>(a.q + r * a.K + k) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
      if ((lane & 7) == 0) a.s[r * a.s_row + (k >> 7) * a.s_kt] = word;
    }
  };
  if (a.positions == nullptr) {
    store(row);
  } else {
    for (int j = 0; j < a.k; ++j) {
      const int p = __shfl_sync(0xFFFFFFFFu, pos, j);
      if (p >= 0 && p < a.R) store(p);
    }
  }
}

// Rows of codes and scale words picked by an index: where rows repeat, cheaper than
// quantising each again (16384 rows of 4096 picked from 2048 tokens, MXFP8 28.0 us in
// one step, 17.9 in two; fp8_128 36.6 and 18.9).  A warp a row, eight rows a CTA, whose
// words of a block of K are one sector.  An index outside [0, T) gives a row of zeros
// with scales of zero.
__global__ void __launch_bounds__(THREADS)
    gather_rows_kernel(const uint8_t* __restrict__ xq, const uint32_t* __restrict__ xs, const int* __restrict__ rows,
                       int64_t T, int64_t R, int64_t K, int KT, uint8_t* __restrict__ q, uint32_t* __restrict__ s) {
  __shared__ int64_t src[THREADS / 32];
  grid_dependency_wait();
  launch_dependents();  // in this order, as above
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * (THREADS / 32), r = r0 + warp;
  int64_t t = r < R ? rows[r] : -1;
  if (t < 0 || t >= T) t = -1;
  if (lane == 0) src[warp] = t;
  __syncthreads();
  {
    const int64_t rw = r0 + (threadIdx.x & 7), tw = src[threadIdx.x & 7];
    for (int kt = threadIdx.x >> 3; kt < KT; kt += THREADS / 8)
      if (rw < R) s[kt * R + rw] = tw < 0 ? 0u : xs[tw * KT + kt];
  }
  if (r >= R) return;
  for (int64_t k0 = lane * 16; k0 < K; k0 += 4 * TASK) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (t >= 0 && k0 + i * TASK < K) v[i] = *reinterpret_cast<const uint4*>(xq + t * K + k0 + i * TASK);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i * TASK < K) *reinterpret_cast<uint4*>(q + r * K + k0 + i * TASK) = v[i];
  }
}

struct ActArgs {
  const __nv_bfloat16* gate;
  const __nv_bfloat16* up;
  int64_t gate_stride, up_stride, K;
  int64_t tasks;
  int segs;
  bool wide;
  uint8_t* q;
  uint32_t* s;
  int64_t s_row, s_kt;
};

// y = gate / (1 + exp(-gate)) * up, quantised: the values of silu_mul_kernel
// (fused_quant.cu), and in MXFP8 its bytes.  Eight CTAs an SM: 4096 x 14336 51.0 us, 53.3
// with the six that 40 registers leave (fp8_128 at 32 registers spills 8 bytes: in the
// 51.0).
template <int FMT>
__global__ void __launch_bounds__(THREADS, 8) silu_mul_rows_kernel(const ActArgs a) {
  grid_dependency_wait();
  launch_dependents();  // in this order, as above
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
  if (task >= a.tasks) return;
  const int64_t row = task / a.segs;
  const int k = static_cast<int>(task - row * a.segs) * TASK + lane * 16;
  uint32_t g[8] = {}, u[8] = {};
  if (k < a.K) {
    load16(a.gate + row * a.gate_stride + k, a.wide, g);
    load16(a.up + row * a.up_stride + k, a.wide, u);
  }
  float y[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float gt = __uint_as_float(j & 1 ? g[j >> 1] & 0xFFFF0000u : g[j >> 1] << 16);
    const float up = __uint_as_float(j & 1 ? u[j >> 1] & 0xFFFF0000u : u[j >> 1] << 16);
    const float e = __expf(-fabsf(gt));
    y[j] = gt * __fdividef(gt >= 0.f ? 1.f : e, 1.f + e) * up;
  }
  uint32_t word;
  Codes c;
  if (FMT == kG8MX) {
    c = quantize16_mx(y, lane, &word);
  } else {
    float s;
    c = quantize16_b128(y, &s);
    word = __float_as_uint(s);
  }
  if (k < a.K) {
    *reinterpret_cast<uint4*>(a.q + row * a.K + k) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
    if ((lane & 7) == 0) a.s[row * a.s_row + (k >> 7) * a.s_kt] = word;
  }
}

// One CTA per 128 x 128 block: row i of the block in lanes 8 (i % 4).. of warp i / 4 % 8.
__global__ void __launch_bounds__(THREADS) quantize_weights_b128_kernel(const __nv_bfloat16* __restrict__ w, int64_t N,
                                                                        int64_t K, int NB, int KT, uint8_t* __restrict__ q,
                                                                        float* __restrict__ s) {
  __shared__ uint32_t top[THREADS / 32];
  const int64_t blk = blockIdx.x;
  const int kt = static_cast<int>(blk % KT);
  const int nb = static_cast<int>(blk / KT % NB);
  const int64_t b = blk / KT / NB;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k = static_cast<int64_t>(kt) * 128 + (lane & 7) * 16;
  uint32_t v[4][8], m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = static_cast<int64_t>(nb) * 128 + i * 32 + warp * 4 + (lane >> 3);
    const bool in = n < N && k < K;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0;
    if (in) load16(w + (b * N + n) * K + k, false, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, v[i][j] & 0x7FFF7FFFu);
  }
  m = max(m & 0xFFFFu, m >> 16);
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (lane == 0) top[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) m = max(m, top[i]);
  const bool nonfinite = m >= 0x7F80u;
  const float amax = __uint_as_float(m << 16);
  float pre;
  const float inv = b128_inverse(amax, &pre);
  if (threadIdx.x == 0) s[blk] = nonfinite ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 448.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = static_cast<int64_t>(nb) * 128 + i * 32 + warp * 4 + (lane >> 3);
    if (n >= N || k >= K) continue;
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = v[i][2 * j + h];
        o |= cvt_e4m3x2(b128_quotient(__uint_as_float(x << 16) * pre, inv),
                        b128_quotient(__uint_as_float(x & 0xFFFF0000u) * pre, inv))
             << (16 * h);
      }
      c[j] = nonfinite ? 0x7F7F7F7Fu : o;
    }
    *reinterpret_cast<uint4*>(q + (b * N + n) * K + k) = make_uint4(c[0], c[1], c[2], c[3]);
  }
}

cudaError_t launch(const void* fn, int64_t blocks, void** args, bool programmatic, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = programmatic ? 1 : 0;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

inline bool is32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

}  // namespace

cudaError_t launch_quantize_rows(const QuantRowsProblem& p, cudaStream_t stream) {
  RowsArgs a;
  a.x = static_cast<const __nv_bfloat16*>(p.x);
  a.rows = p.rows;
  a.positions = p.positions;
  a.k = p.k;
  a.T = p.T;
  a.R = p.R;
  a.K = p.K;
  a.segs = static_cast<int>(ceil_div(p.K, TASK));
  a.tasks = (p.positions != nullptr ? p.T : p.R) * a.segs;
  a.wide = is32(p.x);  // K % 16 == 0: every row then is
  a.q = p.q;
  a.s = static_cast<uint32_t*>(p.s);
  a.s_row = p.s_row;
  a.s_kt = p.s_kt;
  const void* fn = p.fmt == kG8MX ? (p.early ? reinterpret_cast<const void*>(quantize_rows_kernel<kG8MX, true>)
                                             : reinterpret_cast<const void*>(quantize_rows_kernel<kG8MX, false>))
                                  : (p.early ? reinterpret_cast<const void*>(quantize_rows_kernel<kG8B128, true>)
                                             : reinterpret_cast<const void*>(quantize_rows_kernel<kG8B128, false>));
  void* args[] = {&a};
  return launch(fn, ceil_div(a.tasks, THREADS / 32), args, p.early, stream);
}

cudaError_t launch_silu_mul_rows(const ActRowsProblem& p, cudaStream_t stream) {
  ActArgs a;
  a.gate = static_cast<const __nv_bfloat16*>(p.gate);
  a.up = static_cast<const __nv_bfloat16*>(p.up);
  a.gate_stride = p.gate_stride;
  a.up_stride = p.up_stride;
  a.K = p.K;
  a.segs = static_cast<int>(ceil_div(p.K, TASK));
  a.tasks = p.M * a.segs;
  a.wide = is32(p.gate) && is32(p.up) && p.gate_stride % 16 == 0 && p.up_stride % 16 == 0;
  a.q = p.q;
  a.s = static_cast<uint32_t*>(p.s);
  a.s_row = p.s_row;
  a.s_kt = p.s_kt;
  const void* fn = p.fmt == kG8MX ? reinterpret_cast<const void*>(silu_mul_rows_kernel<kG8MX>)
                                  : reinterpret_cast<const void*>(silu_mul_rows_kernel<kG8B128>);
  void* args[] = {&a};
  return launch(fn, ceil_div(a.tasks, THREADS / 32), args, true, stream);
}

cudaError_t launch_gather_rows(const void* xq, const void* xs, const int* rows, int64_t T, int64_t R, int64_t K, uint8_t* q,
                               void* s, cudaStream_t stream) {
  const uint8_t* q0 = static_cast<const uint8_t*>(xq);
  const uint32_t* s0 = static_cast<const uint32_t*>(xs);
  uint32_t* s1 = static_cast<uint32_t*>(s);
  int KT = static_cast<int>(ceil_div(K, 128));
  void* args[] = {&q0, &s0, &rows, &T, &R, &K, &KT, &q, &s1};
  return launch(reinterpret_cast<const void*>(gather_rows_kernel), ceil_div(R, THREADS / 32), args, true, stream);
}

cudaError_t launch_transpose_words(const void* in, int64_t R, int64_t KT, void* out, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(R, 32)), static_cast<unsigned>(ceil_div(KT, 32)), 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, transpose_words_kernel, static_cast<const uint32_t*>(in), R, static_cast<int>(KT),
                            static_cast<uint32_t*>(out));
}

cudaError_t launch_quantize_weights_b128(const void* w, int64_t B, int64_t N, int64_t K, uint8_t* q, float* s,
                                         cudaStream_t stream) {
  const int NB = static_cast<int>(ceil_div(N, 128)), KT = static_cast<int>(ceil_div(K, 128));
  quantize_weights_b128_kernel<<<static_cast<unsigned>(B * NB * KT), THREADS, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(w), N, K, NB, KT, q, s);
  return cudaGetLastError();
}

}  // namespace mx
