// fused_quant.cu - the steps that feed a quantised linear layer, each with its
// output already quantised (MXFP8, MXFP4 or NVFP4; rules in mx_fp4.cuh):
//
//   rmsnorm : t = x + residual (fp32), y = t * rsqrt(mean(t^2) + eps) * w,
//             outputs quantise(y), t rounded once to the residual's type, and
//             optionally y as bf16;
//   silu_mul: y = gate / (1 + exp(-gate)) * up, output quantise(y);
//   fp4     : y = x, the plain 4-bit quantise call;
// the exact widening of packed E2M1 codes to E4M3 bytes, and the repack of
// row-major activation scales into atoms.
//
// y stays in fp32 from the sum to the element's rounding: it is rounded once.
// All read each input once and write each output once, and are bound by HBM
// on long inputs and by one round trip to memory on short ones.
//
// A thread owns chunks of 16 consecutive elements: one NVFP4 block, or half a
// 32-element one, so a block's scale is worked out once or twice.  The scale
// bytes of four blocks are gathered into one word by shuffles (a byte at a time
// into the packed atoms cost the activation 5 us of 52 at 4096 x 14336).
//
// Measured (us, back to back in a CUDA graph; MXFP8 unless named): rmsnorm with
// a bf16 residual 8192 x 4096 34.8 (6.8 TB/s), 4 x 4096 1.7, two chunks a thread
// 2048 x 16384 37.1 (6.4 TB/s), 4 x 16384 3.2, four 1024 x 32768 45.3 (5.2: one
// CTA an SM); silu_mul 4096 x 14336 44.5 (6.6 TB/s), MXFP4 42.2 (6.3), NVFP4 44.5
// (6.0: twice the block scales, each with a reciprocal), 16 x 14336 1.6; fp4 14336
// x 4096 23.2 (6.4 TB/s), NVFP4 23.8 (6.3), 8192 x 14336 to packed scales 43.1
// (6.9), NVFP4 44.9 (6.7); unpack of 14336 x 4096 codes 12.9 (6.8 TB/s).
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
  const float* g;      // NVFP4 tensor scale, or nullptr for 1
  int64_t K;           // elements per row
  int64_t RT;          // packed scales: atom row tiles of a batch,
  uint32_t rows_per_b;  // its rows (0: one batch)
  int64_t b_stride;    // and its bytes
};

QuantOut quant_out(int fmt, uint8_t* q, uint8_t* s, const float* g, int64_t B, int64_t M, int64_t K, bool packed) {
  const int64_t ext = fp4_scale_extent(fmt, K);
  return QuantOut{q, s, g, K, packed ? ceil_div(M, kAtomRows) : 0, B == 1 ? 0u : static_cast<uint32_t>(M), sf_packed_bytes(1, M, ext)};
}

// Chunk c of a row: 32 bytes of bf16 (64 of fp32), as whole sectors when the
// rows start on 32-byte boundaries (wide; uniform over the grid), else as
// 16-byte pieces.
struct Chunk {
  uint32_t w[8];
};

__device__ __forceinline__ Chunk zero_chunk() { return Chunk{{0, 0, 0, 0, 0, 0, 0, 0}}; }

__device__ __forceinline__ Chunk load_32(const void* p, bool wide) {
  Chunk r;
  if (wide) {
    ld_global_32(p, r.w);
  } else {
    const uint4* q = static_cast<const uint4*>(p);
    const uint4 lo = q[0], hi = q[1];
    r = Chunk{{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
  }
  return r;
}

__device__ __forceinline__ void store_32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    st_global_32(p, w);
  } else {
    uint4* q = static_cast<uint4*>(p);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__device__ __forceinline__ Chunk load16(const __nv_bfloat16* row, int c, bool wide) {
  return load_32(row + 16 * static_cast<int64_t>(c), wide);
}

__device__ __forceinline__ void unpack16(const Chunk& v, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = __uint_as_float(v.w[i] << 16);
    f[2 * i + 1] = __uint_as_float(v.w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void store16(__nv_bfloat16* row, int c, const float (&f)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  store_32(row + 16 * static_cast<int64_t>(c), w, wide);
}

// Where a row's codes and scales start.  The quantise and activation kernels work
// it out once a thread, while its loads are in flight: with the offsets and the
// division by the batch's rows at every chunk, 16 x [512, 7168] took 28.3 us
// instead of 25.2 to packed NVFP4, 4096 x 14336 of activation 45.1 instead of 42.7
// to packed MXFP4.
struct OutRow {
  uint8_t* q;
  uint8_t* s;  // packed scales: its word of the first atom along K
};

template <int FMT>
__device__ __forceinline__ OutRow out_row(const QuantOut& o, int64_t row) {
  OutRow r = {o.q + (FMT == kQMX8 ? row * o.K : row * o.K / 2), o.s};
  if (o.RT == 0) {
    r.s += row * (o.K / q_block(FMT));
    return r;
  }
  uint32_t rb = static_cast<uint32_t>(row);  // row of its batch
  if (o.rows_per_b != 0) {
    const uint32_t b = rb / o.rows_per_b;
    rb -= b * o.rows_per_b;
    r.s += b * o.b_stride;
  }
  r.s += static_cast<int64_t>(rb >> 7) * kAtomBytes + (rb & 31) * 16 + ((rb >> 5) & 3) * 4;
  return r;
}

// Quantise chunk `c` (16 elements) of a row and store it.  Every lane of the
// warp calls with consecutive chunks, lane 0's a multiple of 32; only valid lanes
// store.  A row is whole 32-element blocks.
template <int FMT>
__device__ __forceinline__ void quantize_store(const QuantOut& o, const OutRow& at, int c, bool valid,
                                               const float (&y)[16], const TensorScale& ts) {
  uint32_t codes[4];
  const uint32_t sb = quantize_lane16<FMT>(y, ts, codes);
  if (valid) {
    if (FMT == kQMX8)
      reinterpret_cast<uint4*>(at.q)[c] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
    else
      reinterpret_cast<uint2*>(at.q)[c] = make_uint2(codes[0], codes[1]);
  }
  // word: the scale bytes of four consecutive blocks, zero past the row's end
  constexpr int kLanes = q_block(FMT) / 16;  // lanes of a block
  uint32_t word = valid ? sb : 0u;
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, kLanes) << 8;
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * kLanes) << 16;
  if (!valid) return;
  const bool first = c % (4 * kLanes) == 0;  // the first lane of the word
  const int w = c / (4 * kLanes);
  if (o.RT != 0) {
    if (first) *reinterpret_cast<uint32_t*>(at.s + w * o.RT * kAtomBytes) = word;
  } else if ((o.K / q_block(FMT) & 3) == 0) {
    if (first) reinterpret_cast<uint32_t*>(at.s)[w] = word;
  } else if (c % kLanes == 0) {
    at.s[c / kLanes] = static_cast<uint8_t>(sb);
  }
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
  bool wide;        // every row starts on a 32-byte boundary
  QuantOut o;
};

constexpr int kNormThreads = 512;

enum { kResNone = 0, kResBf16 = 1, kResF32 = 2 };

// One CTA per row, the row held in registers (CH chunks a thread) between the
// sum of squares and the output, so x and the residual are read once.  Nothing
// is read before the dependency wait: the weight too may be the output of a
// kernel that let this one start early (an adaptive norm's, from a few-token
// linear layer).  The next kernel in the stream may start at once (it reads
// this one's output after its own wait).
template <int FMT, int CH, int RES>
__global__ void __launch_bounds__(kNormThreads, CH == 1 ? 3 : (CH == 2 ? 2 : 1)) rmsnorm_kernel(const NormArgs a) {
  __shared__ float part[32];
  launch_dependents();
  const int64_t row = blockIdx.x;
  const int nchunks = static_cast<int>(a.o.K / 16);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  // all loads first, so that they are in flight together
  const float g = FMT == kQNV4 && a.o.g != nullptr ? *a.o.g : 1.f;
  Chunk xv[CH], rv[CH][RES == kResF32 ? 2 : 1];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    const bool valid = c < nchunks;
    xv[i] = valid ? load16(a.x + row * a.x_stride, c, a.wide) : zero_chunk();
    if (RES == kResBf16)
      rv[i][0] =
          valid ? load16(static_cast<const __nv_bfloat16*>(a.res) + row * a.res_stride, c, a.wide) : zero_chunk();
    if (RES == kResF32) {
      const float* rp = static_cast<const float*>(a.res) + row * a.res_stride + 16 * static_cast<int64_t>(c);
#pragma unroll
      for (int h = 0; h < (RES == kResF32 ? 2 : 1); ++h) rv[i][h] = valid ? load_32(rp + 8 * h, a.wide) : zero_chunk();
    }
  }
  Chunk w = zero_chunk();
  if (CH == 1) w = static_cast<int>(threadIdx.x) < nchunks ? load16(a.w, threadIdx.x, a.wide) : zero_chunk();
  float t[CH][16];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    unpack16(xv[i], t[i]);
    if (RES == kResBf16) {
      float r[16];
      unpack16(rv[i][0], r);
#pragma unroll
      for (int j = 0; j < 16; ++j) t[i][j] += r[j];
    }
    if (RES == kResF32) {
#pragma unroll
      for (int j = 0; j < 16; ++j) t[i][j] += __uint_as_float(rv[i][RES == kResF32 ? j >> 3 : 0].w[j & 7]);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) ss = fmaf(t[i][j], t[i][j], ss);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  // every warp adds the partials itself, in the same order
  ss = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
  const float rstd = rsqrtf(ss / static_cast<float>(a.o.K) + a.eps);
  const TensorScale ts = tensor_scale(g);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (i > 0 && (c & ~31) >= nchunks) break;  // the whole warp is past the row
    const bool valid = c < nchunks;
    if (RES == kResBf16 && valid) store16(static_cast<__nv_bfloat16*>(a.res_out) + row * a.o.K, c, t[i], a.wide);
    if (RES == kResF32 && valid) {
      float* rp = static_cast<float*>(a.res_out) + row * a.o.K + 16 * static_cast<int64_t>(c);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(t[i][8 * h + j]);
        store_32(rp + 8 * h, r, a.wide);
      }
    }
    float wf[16];
    unpack16(CH == 1 ? w : (valid ? load16(a.w, c, a.wide) : zero_chunk()), wf);
#pragma unroll
    for (int j = 0; j < 16; ++j) t[i][j] = t[i][j] * rstd * wf[j];
    if (a.y != nullptr && valid) store16(a.y + row * a.o.K, c, t[i], a.wide);
    quantize_store<FMT>(a.o, out_row<FMT>(a.o, row), c, valid, t[i], ts);
  }
}

constexpr int kRowThreads = 128;

struct ActArgs {
  const __nv_bfloat16* gate;
  const __nv_bfloat16* up;
  int64_t gate_stride, up_stride;
  int segs;   // CTAs per row
  bool wide;  // every row starts on a 32-byte boundary
  QuantOut o;
};


// A CTA takes CH x blockDim.x chunks of one row (a row is `segs` CTAs).  Twelve
// CTAs an SM, ten for NVFP4, which spills at twelve (4096 x 14336: 46.0 -> 44.1 us;
// MXFP4 at ten 42.2 -> 43.7).
template <int FMT, int CH>
__global__ void __launch_bounds__(kRowThreads, FMT == kQNV4 ? 10 : 12) silu_mul_kernel(const ActArgs a) {
  launch_dependents();
  const int64_t row = blockIdx.x / a.segs;
  const int c0 = static_cast<int>(blockIdx.x - row * a.segs) * (CH * blockDim.x) + threadIdx.x;
  const int nchunks = static_cast<int>(a.o.K / 16);
  grid_dependency_wait();
  Chunk gv[CH], uv[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + i * blockDim.x;
    gv[i] = c < nchunks ? load16(a.gate + row * a.gate_stride, c, a.wide) : zero_chunk();
    uv[i] = c < nchunks ? load16(a.up + row * a.up_stride, c, a.wide) : zero_chunk();
  }
  const OutRow at = out_row<FMT>(a.o, row);
  const TensorScale ts = tensor_scale(FMT == kQNV4 && a.o.g != nullptr ? *a.o.g : 1.f);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + i * blockDim.x;
    if ((c & ~31) >= nchunks) return;  // the whole warp is past the row
    float gt[16], up[16];
    unpack16(gv[i], gt);
    unpack16(uv[i], up);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      // gate / (1 + exp(-gate)) with the exponential's argument <= 0, so that
      // nothing overflows and very negative gates keep their value.  The quick
      // exponential and division are off by 2 + 1.2 |gate| and 2 ulp, 1e-5 at
      // |gate| = 64 and far below an 8-bit element's half step (2^-4); with the
      // accurate ones NVFP4 4096 x 14336 takes 73.5 us instead of 44.5.
      const float e = __expf(-fabsf(gt[j]));
      gt[j] = gt[j] * __fdividef(gt[j] >= 0.f ? 1.f : e, 1.f + e) * up[j];
    }
    quantize_store<FMT>(a.o, at, c, c < nchunks, gt, ts);
  }
}

struct Fp4Args {
  const __nv_bfloat16* x;  // dense rows
  int segs;                // CTAs per row
  bool wide;
  QuantOut o;
};

// kEarly as in quantize.cu: only the activation quantise inside a linear call
// lets the next kernel start early, never the call that may make weights.
template <int FMT, bool kEarly, int CH>
__global__ void __launch_bounds__(kRowThreads, CH == 1 ? 12 : 10) quantize_fp4_kernel(const Fp4Args a) {
  if (kEarly) {
    launch_dependents();
    grid_dependency_wait();
  }
  const int64_t row = blockIdx.x / a.segs;
  const int c0 = static_cast<int>(blockIdx.x - row * a.segs) * (CH * blockDim.x) + threadIdx.x;
  const int nchunks = static_cast<int>(a.o.K / 16);
  Chunk v[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + i * blockDim.x;
    v[i] = c < nchunks ? load16(a.x + row * a.o.K, c, a.wide) : zero_chunk();
  }
  const OutRow at = out_row<FMT>(a.o, row);
  const TensorScale ts = tensor_scale(FMT == kQNV4 && a.o.g != nullptr ? *a.o.g : 1.f);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + i * blockDim.x;
    if ((c & ~31) >= nchunks) return;  // the whole warp is past the row
    float x[16];
    unpack16(v[i], x);
    quantize_store<FMT>(a.o, at, c, c < nchunks, x, ts);
  }
}

// Four E2M1 codes (the low 16 bits of w) -> four E4M3 bytes, a table lookup by
// byte permute; the signs move from bit 3 of a nibble to bit 7 of a byte.
__device__ __forceinline__ uint32_t e2m1x4_to_e4m3(uint32_t w) {
  const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, w & 0x7777u);
  const uint32_t sign = ((w & 0x8u) << 4) | ((w & 0x80u) << 8) | ((w & 0x800u) << 12) | ((w & 0x8000u) << 16);
  return mag | sign;
}

// 16 codes a lane: 8 bytes in, 16 out, both contiguous over the warp.
__global__ void __launch_bounds__(256) fp4_unpack_kernel(const uint2* __restrict__ q, uint4* __restrict__ out,
                                                         uint64_t n) {
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const uint2 v = __ldg(q + i);
  out[i] = make_uint4(e2m1x4_to_e4m3(v.x), e2m1x4_to_e4m3(v.x >> 16), e2m1x4_to_e4m3(v.y), e2m1x4_to_e4m3(v.y >> 16));
}

// Row-major scales [B, R, KB] -> packed atoms, for pre-quantised activations.  A
// CTA turns 128 rows x 32 bytes into 8 atoms through shared memory, so that both
// sides move whole sectors (V bytes a load, KB % V == 0).
constexpr int kRepackThreads = 256;

template <int V>
__global__ void __launch_bounds__(kRepackThreads) sf_repack_kernel(const uint8_t* __restrict__ src, int64_t R, int KB,
                                                                   int KT, int RT, uint8_t* __restrict__ dst) {
  __shared__ uint32_t tile[kAtomRows][9];  // 8 words a row, one of padding
  launch_dependents();
  grid_dependency_wait();
  const int kt0 = blockIdx.x * 8, rt = blockIdx.y;
  const int64_t b = blockIdx.z;
  constexpr int kPieces = 32 / V;
  for (int p = threadIdx.x; p < kAtomRows * kPieces; p += kRepackThreads) {
    const int r = p / kPieces, o = p % kPieces * V;
    const int64_t row = static_cast<int64_t>(rt) * kAtomRows + r;
    const int byte = kt0 * 4 + o;
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) w[i] = 0;
    if (row < R && byte < KB) {
      const uint8_t* s = src + (b * R + row) * KB + byte;
      if constexpr (V == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(s);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(s);
      }
    }
#pragma unroll
    for (int i = 0; i < V / 4; ++i) tile[r][o / 4 + i] = w[i];
  }
  __syncthreads();
  const int a = threadIdx.x >> 5, l = threadIdx.x & 31;
  if (kt0 + a < KT)
    *reinterpret_cast<uint4*>(dst + ((b * KT + kt0 + a) * RT + rt) * kAtomBytes + l * 16) =
        make_uint4(tile[l][a], tile[l + 32][a], tile[l + 64][a], tile[l + 96][a]);
}

cudaError_t launch_pdl(const void* kern, int64_t grid, int threads, void* args, cudaStream_t stream,
                       bool programmatic = true) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = programmatic ? 1 : 0;
  void* params[1] = {args};
  return cudaLaunchKernelExC(&cfg, kern, params);
}

// Chunks a thread, threads and CTAs for M rows of K elements, the CTAs of a row
// as even as whole warps allow.  `most` chunks a thread keep more bytes in
// flight on long inputs (4-bit quantise, 14336 x 4096: 23.9 -> 23.2 us, NVFP4 28.3
// -> 23.8; activation, 4096 x 14336 to MXFP8 48.9 -> 44.5) and one starts more CTAs
// on short ones (activation, 512 x 14336: 7.0 -> 6.6 us).
int row_split(int64_t M, int64_t K, int most, int* threads, int* segs) {
  const int64_t chunks = K / 16;
  const int ch = chunks >= 32 * most && M * chunks >= 152ll * 32 * 2 * kRowThreads ? most : 1;
  *segs = static_cast<int>(ceil_div(chunks, ch * kRowThreads));
  *threads = static_cast<int>(ceil_div(ceil_div(chunks, *segs * ch), 32) * 32);
  return ch;
}

// Whether rows of `elem`-byte elements at p, `stride` elements apart, all start
// on 32-byte boundaries (absent tensors do).
bool rows_32(const void* p, int64_t stride, int elem) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 32 == 0 && stride * elem % 32 == 0);
}

template <int FMT>
const void* act_kernel(int ch) {
  return ch == 2 ? reinterpret_cast<const void*>(silu_mul_kernel<FMT, 2>)
                 : reinterpret_cast<const void*>(silu_mul_kernel<FMT, 1>);
}

template <int FMT>
const void* fp4_kernel(bool early, int ch) {
  if (early)
    return ch == 4 ? reinterpret_cast<const void*>(quantize_fp4_kernel<FMT, true, 4>)
                   : reinterpret_cast<const void*>(quantize_fp4_kernel<FMT, true, 1>);
  return ch == 4 ? reinterpret_cast<const void*>(quantize_fp4_kernel<FMT, false, 4>)
                 : reinterpret_cast<const void*>(quantize_fp4_kernel<FMT, false, 1>);
}

template <int FMT, int CH>
void* norm_kernel(int res) {
  return res == kResNone ? reinterpret_cast<void*>(rmsnorm_kernel<FMT, CH, kResNone>)
                         : (res == kResBf16 ? reinterpret_cast<void*>(rmsnorm_kernel<FMT, CH, kResBf16>)
                                            : reinterpret_cast<void*>(rmsnorm_kernel<FMT, CH, kResF32>));
}

template <int FMT>
void* norm_kernel(int ch, int res) {
  return ch == 1 ? norm_kernel<FMT, 1>(res) : (ch == 2 ? norm_kernel<FMT, 2>(res) : norm_kernel<FMT, 4>(res));
}

}  // namespace

cudaError_t launch_rmsnorm_quantize(const NormProblem& p, cudaStream_t stream) {
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
  a.o = quant_out(p.fmt, p.q, p.s, p.g, 1, p.M, p.K, p.packed);
  const int re = p.res_f32 ? 4 : 2;
  a.wide = rows_32(p.x, p.x_stride, 2) && rows_32(p.res, p.res_stride, re) && rows_32(p.res_out, p.K, re) &&
           rows_32(p.w, 0, 2) && rows_32(p.y, p.K, 2);
  const int res = p.res == nullptr ? kResNone : (p.res_f32 ? kResF32 : kResBf16);
  const int64_t chunks = p.K / 16;
  // one chunk a thread while that fits a CTA
  int ch = 1;
  while (ceil_div(chunks, ch) > kNormThreads) ch *= 2;
  if (ch > 4) return cudaErrorInvalidValue;  // the host refuses these first
  const int threads = static_cast<int>(ceil_div(ceil_div(chunks, ch), 32) * 32);
  void* k = p.fmt == kQMX8 ? norm_kernel<kQMX8>(ch, res)
                           : (p.fmt == kQMX4 ? norm_kernel<kQMX4>(ch, res) : norm_kernel<kQNV4>(ch, res));
  return launch_pdl(k, p.M, threads, &a, stream);
}

cudaError_t launch_silu_mul_quantize(const ActProblem& p, cudaStream_t stream) {
  if (p.M == 0) return cudaSuccess;
  ActArgs a;
  a.gate = static_cast<const __nv_bfloat16*>(p.gate);
  a.up = static_cast<const __nv_bfloat16*>(p.up);
  a.gate_stride = p.gate_stride;
  a.up_stride = p.up_stride;
  a.o = quant_out(p.fmt, p.q, p.s, p.g, 1, p.M, p.K, p.packed);
  a.wide = rows_32(p.gate, p.gate_stride, 2) && rows_32(p.up, p.up_stride, 2);
  int threads;
  const int ch = row_split(p.M, p.K, 2, &threads, &a.segs);
  const int64_t grid = p.M * a.segs;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;  // the host refuses these first
  const void* k = p.fmt == kQMX8 ? act_kernel<kQMX8>(ch) : (p.fmt == kQMX4 ? act_kernel<kQMX4>(ch) : act_kernel<kQNV4>(ch));
  return launch_pdl(k, grid, threads, &a, stream);
}

cudaError_t launch_quantize_fp4(int fmt, const void* x, int64_t B, int64_t M, int64_t K, const float* g, uint8_t* q,
                                uint8_t* s, bool packed_scales, cudaStream_t stream, bool early_trigger) {
  if (B * M == 0) return cudaSuccess;
  Fp4Args a;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.wide = rows_32(x, K, 2);
  a.o = quant_out(fmt, q, s, g, B, M, K, packed_scales);
  int threads;
  const int ch = row_split(B * M, K, 4, &threads, &a.segs);
  const int64_t grid = B * M * a.segs;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;  // the host refuses these first
  const void* k = fmt == kQNV4 ? fp4_kernel<kQNV4>(early_trigger, ch) : fp4_kernel<kQMX4>(early_trigger, ch);
  return launch_pdl(k, grid, threads, &a, stream, early_trigger);
}

cudaError_t launch_sf_repack(const uint8_t* src, int64_t B, int64_t R, int64_t KB, uint8_t* dst, cudaStream_t stream) {
  const int64_t RT = ceil_div(R, kAtomRows), KT = ceil_div(KB, 4);
  if (KB % 4 != 0 || RT > 65535 || B > 65535) return cudaErrorInvalidValue;  // the caller takes sf_pack then
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(KT, 8)), static_cast<unsigned>(RT), static_cast<unsigned>(B));
  cfg.blockDim = dim3(kRepackThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto k = KB % 16 == 0 ? sf_repack_kernel<16> : sf_repack_kernel<4>;
  return cudaLaunchKernelEx(&cfg, k, src, R, static_cast<int>(KB), static_cast<int>(KT), static_cast<int>(RT), dst);
}

cudaError_t launch_fp4_unpack(const uint8_t* q, int64_t n, uint8_t* out, cudaStream_t stream) {
  const int64_t chunks = n / 16, grid = ceil_div(chunks, 256);
  if (grid == 0) return cudaSuccess;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;  // the host refuses these first
  fp4_unpack_kernel<<<static_cast<unsigned>(grid), 256, 0, stream>>>(
      reinterpret_cast<const uint2*>(q), reinterpret_cast<uint4*>(out), static_cast<uint64_t>(chunks));
  return cudaGetLastError();
}

}  // namespace mx
