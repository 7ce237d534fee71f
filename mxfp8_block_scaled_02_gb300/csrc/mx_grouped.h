// mx_grouped.h - launchers of the grouped and block-128 products, the quantising
// steps that feed them, and the expert routing.  Internal: not part of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mx {

// Formats (MXFP8_GFMT_*)
constexpr int kG8MX = 0;    // E4M3, one E8M0 scale per 32 along K
constexpr int kG8B128 = 1;  // E4M3, one fp32 scale per 128 along K (x) or per 128 x 128 (weights)

constexpr int kMaxGroups = 512;

// gemm_grouped.cu: out[r] = x[r] w[e]^T + bias[e] for r in [offsets[e], offsets[e + 1]),
// or, with offsets null, r in [e R / E, (e + 1) R / E).
struct GroupedProblem {
  int fmt;
  const uint8_t* x;       // E4M3 [R, K]
  const void* xs;         // scales of x, one 4-byte word per row and 128 of K (four E8M0
  int64_t xs_row, xs_kt;  // bytes, or one fp32): strides in words
  const uint8_t* w;       // E4M3 [E, N, K]
  const void* ws;         // packed atoms (MXFP8), or fp32 [E, ceil(N / 128), ceil(K / 128)]
  const void* bias;       // bf16, or nullptr
  int64_t bias_stride;    // elements between two groups' biases (0: one for all)
  void* out;              // bf16 [R, N]
  const int* offsets;     // device, [E + 1], or nullptr
  int64_t E, R, N, K;
  // 1: the kernel before this one in the stream does not write the offsets and lets
  // this one start only when all before it is done (the kernels of grouped_quant.cu):
  // offsets, weights and their scales are read without waiting for it
  int offsets_ready = 0;
  // b128_quantizes_inside: bf16 x [R, K] instead of x and xs
  const void* x_bf16 = nullptr;
};
// How a shape is run: a CTA pair (cg = 2) or one CTA a tile, the rows of x a tile
// takes at most, and the K splits.
struct GroupedPlan {
  int cg, tn, splits;
};
// Whether fp8_128 products of bf16 x quantise it in their own kernel: few rows, no groups.
bool b128_quantizes_inside(bool ragged, int64_t E, int64_t R);
GroupedPlan grouped_plan(int fmt, int64_t E, int64_t R, int64_t N, int64_t K, bool ragged);
// Tiles of up to tn rows of x that R rows in E groups can come to.
int64_t grouped_max_tiles(int64_t E, int64_t R, bool ragged, int tn);
cudaError_t launch_gemm_grouped(const GroupedProblem& p, const GroupedPlan& plan, int sms, cudaStream_t stream,
                                const char** msg);
cudaError_t take_status_grouped(unsigned int* out);
// gemm_b128_pair.cu: fp8_128 on CTA pairs.
cudaError_t launch_gemm_b128_pair(const GroupedProblem& p, int sms, cudaStream_t stream, const char** msg);
cudaError_t take_status_b128_pair(unsigned int* out);

// grouped_quant.cu.  Row r of the output is x[rows[r]] (rows null: x[r]), a row
// index outside [0, T) gives zeros; or, with positions, row t of x goes to the rows
// positions[t][0 .. k) that are in [0, R) (read once, written k times).  Codes [R, K]; the scales' 4-byte words (as
// GroupedProblem::xs) at r * s_row + kt * s_kt.
struct QuantRowsProblem {
  int fmt;
  const void* x;         // bf16 [T, K]
  const int* rows;       // device [R], or nullptr
  int64_t T, R, K;
  uint8_t* q;
  void* s;
  int64_t s_row, s_kt;
  bool early;            // let the next kernel in the stream start before this one ends
  const int* positions = nullptr;  // device [T, k]; rows null
  int k = 0;                       // at most 32
};
cudaError_t launch_quantize_rows(const QuantRowsProblem& p, cudaStream_t stream);
// silu(gate) * up with the output quantised; rows of 16-byte aligned bf16.  Lets the
// next kernel in the stream start early.
struct ActRowsProblem {
  int fmt;
  const void* gate;
  int64_t gate_stride;
  const void* up;
  int64_t up_stride;
  int64_t M, K;
  uint8_t* q;
  void* s;
  int64_t s_row, s_kt;
};
cudaError_t launch_silu_mul_rows(const ActRowsProblem& p, cudaStream_t stream);
// Codes [T, K] and scale words [T][KT] -> those of rows [R], words as [KT][R]; a row of
// zeros for an index outside [0, T).
cudaError_t launch_gather_rows(const void* xq, const void* xs, const int* rows, int64_t T, int64_t R, int64_t K, uint8_t* q,
                               void* s, cudaStream_t stream);
// Scale words [R][KT] -> [KT][R] (KT at most 2^21).
cudaError_t launch_transpose_words(const void* in, int64_t R, int64_t KT, void* out, cudaStream_t stream);
// bf16 weights [B, N, K] -> E4M3 codes and fp32 scales [B, ceil(N / 128), ceil(K / 128)].
cudaError_t launch_quantize_weights_b128(const void* w, int64_t B, int64_t N, int64_t K, uint8_t* q, float* s,
                                         cudaStream_t stream);

// route.cu
constexpr int kRouteMaxE = 512;
constexpr int kRouteMaxK = 32;
struct RouteProblem {
  const void* logits;  // [T, E] rows
  int64_t stride;      // elements
  int bf16;            // 1: bf16 logits, 0: fp32
  int64_t T;
  int E, k;
  int sigmoid;         // 1: weights sigmoid(logit), 0: softmax over all E
  int renormalize;
  float scale;
  int* ids;            // [T, k]
  float* weights;      // [T, k]
  int* offsets;        // [E + 1]
  int* rows;           // [T k]
  int* positions;      // [T, k]
  int* counts;         // workspace, route_count_bytes
};
int64_t route_count_bytes(int64_t T, int E);
cudaError_t launch_route(const RouteProblem& p, cudaStream_t stream);
struct CombineProblem {
  const void* y;         // bf16 [R, N]
  const int* positions;  // [T, k]
  const float* weights;  // [T, k]
  const void* add;       // bf16 [T, N] rows, or nullptr
  int64_t add_stride;
  int64_t T, R, N;
  int k;
  void* out;             // bf16 [T, N]
};
cudaError_t launch_combine(const CombineProblem& p, cudaStream_t stream);

}  // namespace mx
