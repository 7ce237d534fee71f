// api_fp4.cu - the C ABI of the 4-bit linear layer and of the fused norm and
// activation steps (declared in include/mxfp8.h).  Host side only: argument
// checks (all before any launch), workspace carving and the choice of kernels.
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_api.h"
#include "mx_fp4.cuh"
#include "mx_kernels.h"
#include "mx_layout.cuh"

static_assert(MXFP8_QFMT_MXFP8 == mx::kQMX8 && MXFP8_QFMT_MXFP4 == mx::kQMX4 && MXFP8_QFMT_NVFP4 == mx::kQNV4,
              "format codes");

namespace {

using mx::aligned;
using mx::cuda_fail;
using mx::fail;
using mx::fp4_scale_extent;
using mx::round_up;

cudaStream_t as_stream(mxfp8_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

mxfp8_status check_fp4(int fmt) {
  if (fmt != MXFP8_QFMT_MXFP4 && fmt != MXFP8_QFMT_NVFP4)
    return fail(MXFP8_ERR_INVALID_ARG, "format %d is not a 4-bit format", fmt);
  return MXFP8_OK;
}

mxfp8_status check_tensor_scale(int fmt, const float* g) {
  if (g != nullptr && fmt != MXFP8_QFMT_NVFP4)
    return fail(MXFP8_ERR_INVALID_ARG, "a tensor scale belongs to NVFP4 only");
  if (!aligned(g, 4)) return fail(MXFP8_ERR_INVALID_ARG, "the tensor scale must be 4-byte aligned");
  return MXFP8_OK;
}

// Sizes of a [B, R, K] tensor of 4-bit (or MXFP8) blocks.
mxfp8_status check_blocks(int fmt, int64_t B, int64_t R, int64_t K, const char* what) {
  if (B < 1 || R < 0 || K < 1)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: B=%lld rows=%lld K=%lld", what, (long long)B, (long long)R, (long long)K);
  if (K % 32 != 0) return fail(MXFP8_ERR_INVALID_ARG, "%s: K=%lld is not a multiple of 32", what, (long long)K);
  if (K > (1ll << 29)) return fail(MXFP8_ERR_UNSUPPORTED, "%s: K=%lld is too large", what, (long long)K);
  return R > 0 ? mx::check_block_count(B, R, fp4_scale_extent(fmt, K), what) : MXFP8_OK;
}

mxfp8_status quantize_impl(int fmt, const void* x, int64_t B, int64_t M, int64_t K, const float* g, uint8_t* q,
                           uint8_t* s, bool packed, mxfp8_stream_t stream) {
  mxfp8_status st = check_fp4(fmt);
  if (st != MXFP8_OK || (st = check_blocks(fmt, B, M, K, "4-bit quantise")) != MXFP8_OK ||
      (st = check_tensor_scale(fmt, g)) != MXFP8_OK)
    return st;
  if (M == 0) return MXFP8_OK;
  if (x == nullptr || q == nullptr || s == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(s, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "x, codes and scales must be 16-byte aligned");
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  cudaError_t e = mx::launch_quantize_fp4(fmt, x, B, M, K, g, q, s, packed, as_stream(stream), false);
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "4-bit quantise launch");
}

// K splits of the CTA-pair kernel that meet in workspace partials (else 1).
int product_splits(int64_t B, int64_t M, int64_t N, int64_t K) {
  return mx::fp4_use_small(B, M, N, K) ? 1 : mx::fp4_splitk_splits(B, M, N, K);
}

// Workspace of a call: codes and packed scales of x (bf16 x; the scales also
// for row-major x_scale), then the split-K partials.
struct WsLayout {
  int64_t xq, sfx, part, total;
};

WsLayout workspace_layout(int fmt, int64_t B, int64_t M, int64_t N, int64_t K, bool have_codes, bool have_atoms,
                          int splits) {
  WsLayout w;
  w.xq = 0;
  w.sfx = have_codes ? 0 : round_up(B * M * K / 2, 256);
  w.part = w.sfx + (have_atoms ? 0 : round_up(mx::sf_packed_bytes(B, M, fp4_scale_extent(fmt, K)), 256));
  w.total = w.part + (splits > 1 ? round_up(4 * splits * B * M * N, 256) : 0);
  return w;
}

mxfp8_status check_product(int fmt, int64_t B, int64_t M, int64_t N, int64_t K) {
  mxfp8_status st = check_fp4(fmt);
  if (st != MXFP8_OK || (st = check_blocks(fmt, B, M, K, "activations")) != MXFP8_OK) return st;
  if (N < 1) return fail(MXFP8_ERR_INVALID_ARG, "N=%lld", (long long)N);
  if (N % 8 != 0) return fail(MXFP8_ERR_UNSUPPORTED, "N=%lld: this library needs N %% 8 == 0", (long long)N);
  if (N > (1ll << 30)) return fail(MXFP8_ERR_UNSUPPORTED, "N=%lld is too large", (long long)N);
  if ((st = check_blocks(fmt, B, N, K, "weights")) != MXFP8_OK) return st;
  // output tiles are counted in 31 bits (tiles are 256 x 256, splits at most 8)
  if (mx::ceil_div(M, 256) * mx::ceil_div(N, 256) > (1ll << 27) / B)
    return fail(MXFP8_ERR_UNSUPPORTED, "B=%lld M=%lld N=%lld has too many output tiles", (long long)B, (long long)M,
                (long long)N);
  return MXFP8_OK;
}

struct Operands {
  const uint8_t* x;    // codes
  const uint8_t* sfx;  // packed atoms
  const float* gx;
  const uint8_t* w;
  const uint8_t* sfw;
  const float* gw;
  const void* bias;
  void* out;
};

mxfp8_status check_operands(int fmt, const Operands& o) {
  if (o.w == nullptr || o.sfw == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null weight pointer");
  if (o.out == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null output pointer");
  if (!aligned(o.x, 16) || !aligned(o.sfx, 16) || !aligned(o.w, 16) || !aligned(o.sfw, 16) || !aligned(o.bias, 16) ||
      !aligned(o.out, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  mxfp8_status st = check_tensor_scale(fmt, o.gx);
  return st == MXFP8_OK ? check_tensor_scale(fmt, o.gw) : st;
}

mxfp8_status run_product(int fmt, const Operands& o, int64_t B, int64_t M, int64_t N, int64_t K, float* part,
                         int splits, int sms, mxfp8_stream_t stream) {
  mx::Fp4Problem p{fmt, o.x, o.w, o.sfx, o.sfw, o.gx, o.gw, o.bias, o.out, B, M, N, K};
  p.part = part;
  p.splits = splits;
  const char* msg = "";
  cudaError_t e = mx::fp4_use_small(B, M, N, K) ? mx::launch_gemm_fp4_small(p, sms, as_stream(stream), &msg)
                                  : mx::launch_gemm_fp4(p, sms, as_stream(stream), &msg);
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, msg);
}

mxfp8_status check_qfmt(int fmt) {
  if (fmt != MXFP8_QFMT_MXFP8 && fmt != MXFP8_QFMT_MXFP4 && fmt != MXFP8_QFMT_NVFP4)
    return fail(MXFP8_ERR_INVALID_ARG, "format %d", fmt);
  return MXFP8_OK;
}

mxfp8_status check_rows(const char* what, const void* p, int64_t stride, int64_t M, int64_t K, int elem_bytes) {
  if (p == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned(p, 16) || (M > 1 && stride * elem_bytes % 16 != 0))
    return fail(MXFP8_ERR_INVALID_ARG, "%s: rows must start on 16-byte boundaries (stride %lld)", what,
                (long long)stride);
  if (M > 1 && stride < K && stride != 0)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: row stride %lld is below K=%lld", what, (long long)stride, (long long)K);
  return MXFP8_OK;
}

}  // namespace

extern "C" {

mxfp8_status mxfp8_fp4_quantize(int fmt, const void* x_bf16, int64_t rows, int64_t K, const float* tensor_scale,
                                uint8_t* x_q, uint8_t* x_scale, mxfp8_stream_t stream) {
  return quantize_impl(fmt, x_bf16, 1, rows, K, tensor_scale, x_q, x_scale, false, stream);
}

mxfp8_status mxfp8_fp4_quantize_packed(int fmt, const void* x_bf16, int64_t B, int64_t M, int64_t K,
                                       const float* tensor_scale, uint8_t* x_q, uint8_t* sfa_packed,
                                       mxfp8_stream_t stream) {
  return quantize_impl(fmt, x_bf16, B, M, K, tensor_scale, x_q, sfa_packed, true, stream);
}

mxfp8_status mxfp8_fp4_unpack(const uint8_t* q, int64_t n, uint8_t* out_e4m3, mxfp8_stream_t stream) {
  if (n < 0 || n % 32 != 0) return fail(MXFP8_ERR_INVALID_ARG, "n=%lld is not a multiple of 32", (long long)n);
  if (n == 0) return MXFP8_OK;
  if (q == nullptr || out_e4m3 == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(q, 16) || !aligned(out_e4m3, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "codes and output must be 16-byte aligned");
  int sms = 0;
  mxfp8_status st = mx::current_device(&sms);
  if (st != MXFP8_OK) return st;
  cudaError_t e = mx::launch_fp4_unpack(q, n, out_e4m3, as_stream(stream));
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "4-bit unpack launch");
}

mxfp8_status mxfp8_fp4_packed_sizes(int fmt, int64_t B, int64_t N, int64_t K, size_t* w_bytes, size_t* sf_bytes) {
  if (w_bytes == nullptr || sf_bytes == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null output pointer");
  mxfp8_status st = check_fp4(fmt);
  if (st != MXFP8_OK) return st;
  if (N < 1) return fail(MXFP8_ERR_INVALID_ARG, "N=%lld", (long long)N);
  if ((st = check_blocks(fmt, B, N, K, "packed sizes")) != MXFP8_OK) return st;
  *w_bytes = static_cast<size_t>(B * N * K / 2);
  *sf_bytes = static_cast<size_t>(mx::sf_packed_bytes(B, N, fp4_scale_extent(fmt, K)));
  return MXFP8_OK;
}

mxfp8_status mxfp8_fp4_process_weights(int fmt, const uint8_t* w, const uint8_t* w_scale, int64_t B, int64_t N,
                                       int64_t K, uint8_t* w_packed, uint8_t* sf_packed, mxfp8_stream_t stream) {
  mxfp8_status st = check_fp4(fmt);
  if (st != MXFP8_OK) return st;
  if (N < 1) return fail(MXFP8_ERR_INVALID_ARG, "N=%lld", (long long)N);
  if ((st = check_blocks(fmt, B, N, K, "weights")) != MXFP8_OK) return st;
  if (w == nullptr || w_scale == nullptr || w_packed == nullptr || sf_packed == nullptr)
    return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(w, 16) || !aligned(w_scale, 16) || !aligned(w_packed, 16) || !aligned(sf_packed, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "weight and scale pointers must be 16-byte aligned");
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  cudaError_t e;
  if (w_packed != w &&
      (e = cudaMemcpyAsync(w_packed, w, static_cast<size_t>(B * N * K / 2), cudaMemcpyDeviceToDevice,
                           as_stream(stream))) != cudaSuccess)
    return cuda_fail(e, "weight copy");
  e = mx::launch_sf_pack(w_scale, B, N, fp4_scale_extent(fmt, K), sf_packed, sms, as_stream(stream), false);
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "scale repack launch");
}

mxfp8_status mxfp8_fp4_workspace_size(int fmt, int64_t B, int64_t M, int64_t N, int64_t K, int x_is_quantized,
                                      size_t* bytes) {
  if (bytes == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null output pointer");
  mxfp8_status st = check_product(fmt, B, M, N, K);
  if (st != MXFP8_OK) return st;
  if (x_is_quantized == 0 && mx::fp4_quantizes_inside(B, M)) {
    *bytes = 0;
    return MXFP8_OK;
  }
  *bytes = static_cast<size_t>(
      workspace_layout(fmt, B, M, N, K, x_is_quantized != 0, false, product_splits(B, M, N, K)).total);
  return MXFP8_OK;
}

mxfp8_status mxfp8_fp4_product_workspace_size(int fmt, int64_t B, int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (bytes == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null output pointer");
  mxfp8_status st = check_product(fmt, B, M, N, K);
  if (st != MXFP8_OK) return st;
  *bytes = static_cast<size_t>(workspace_layout(fmt, B, M, N, K, true, true, product_splits(B, M, N, K)).total);
  return MXFP8_OK;
}

mxfp8_status mxfp8_fp4_linear(int fmt, const void* x_bf16, const uint8_t* x_q, const uint8_t* x_scale,
                              const float* x_tensor_scale, int64_t B, int64_t M, int64_t N, int64_t K,
                              const uint8_t* w_packed, const uint8_t* sf_packed, const float* w_tensor_scale,
                              const void* bias_bf16, void* out_bf16, void* workspace, size_t workspace_bytes,
                              mxfp8_stream_t stream) {
  mxfp8_status st = check_product(fmt, B, M, N, K);
  if (st != MXFP8_OK) return st;
  if (M == 0) return MXFP8_OK;
  const bool have_x = x_bf16 != nullptr, have_q = x_q != nullptr || x_scale != nullptr;
  if (have_x == have_q) return fail(MXFP8_ERR_INVALID_ARG, "pass exactly one of x_bf16 or (x_q, x_scale)");
  if (have_q && (x_q == nullptr || x_scale == nullptr))
    return fail(MXFP8_ERR_INVALID_ARG, "x_q and x_scale must both be given");
  Operands o{x_q, x_scale, x_tensor_scale, w_packed, sf_packed, w_tensor_scale, bias_bf16, out_bf16};
  if ((st = check_operands(fmt, o)) != MXFP8_OK) return st;
  if (!aligned(x_bf16, 16)) return fail(MXFP8_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  int sms = 0;
  if (have_x && mx::fp4_quantizes_inside(B, M)) {
    if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
    mx::Fp4Problem p{fmt, nullptr, o.w, nullptr, o.sfw, o.gx, o.gw, o.bias, o.out, B, M, N, K};
    p.x_bf16 = x_bf16;
    const char* msg = "";
    cudaError_t e = mx::launch_gemm_fp4_small(p, sms, as_stream(stream), &msg);
    return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, msg);
  }
  const int splits = product_splits(B, M, N, K);
  const WsLayout ws = workspace_layout(fmt, B, M, N, K, have_q, false, splits);
  if (static_cast<int64_t>(workspace_bytes) < ws.total)
    return fail(MXFP8_ERR_INVALID_ARG, "workspace has %zu bytes, needs %lld", workspace_bytes, (long long)ws.total);
  if (workspace == nullptr || !aligned(workspace, 256))
    return fail(MXFP8_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  cudaError_t e;
  if (have_x) {
    e = mx::launch_quantize_fp4(fmt, x_bf16, B, M, K, x_tensor_scale, wsb + ws.xq, wsb + ws.sfx, true, as_stream(stream),
                                true);
    o.x = wsb + ws.xq;
  } else {
    const int64_t KB = K / mx::q_block(fmt);
    e = KB % 4 == 0 && B <= 65535 && M <= 65535 * mx::kAtomRows
            ? mx::launch_sf_repack(x_scale, B, M, KB, wsb + ws.sfx, as_stream(stream))
            : mx::launch_sf_pack(x_scale, B, M, fp4_scale_extent(fmt, K), wsb + ws.sfx, sms, as_stream(stream), true);
  }
  if (e != cudaSuccess) return cuda_fail(e, have_x ? "4-bit quantise launch" : "activation scale repack launch");
  o.sfx = wsb + ws.sfx;
  return run_product(fmt, o, B, M, N, K, splits > 1 ? reinterpret_cast<float*>(wsb + ws.part) : nullptr, splits, sms,
                     stream);
}

mxfp8_status mxfp8_fp4_gemm_packed(int fmt, const uint8_t* x_q, const uint8_t* sfa_packed, const float* x_tensor_scale,
                                   int64_t B, int64_t M, int64_t N, int64_t K, const uint8_t* w_packed,
                                   const uint8_t* sf_packed, const float* w_tensor_scale, const void* bias_bf16,
                                   void* out_bf16, void* workspace, size_t workspace_bytes, mxfp8_stream_t stream) {
  mxfp8_status st = check_product(fmt, B, M, N, K);
  if (st != MXFP8_OK) return st;
  if (M == 0) return MXFP8_OK;
  if (x_q == nullptr || sfa_packed == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  const Operands o{x_q, sfa_packed, x_tensor_scale, w_packed, sf_packed, w_tensor_scale, bias_bf16, out_bf16};
  if ((st = check_operands(fmt, o)) != MXFP8_OK) return st;
  int splits = product_splits(B, M, N, K);
  const WsLayout ws = workspace_layout(fmt, B, M, N, K, true, true, splits);
  if (workspace != nullptr && !aligned(workspace, 256))
    return fail(MXFP8_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace == nullptr || static_cast<int64_t>(workspace_bytes) < ws.total) splits = 1;
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  return run_product(fmt, o, B, M, N, K, splits > 1 ? static_cast<float*>(workspace) : nullptr, splits, sms, stream);
}

mxfp8_status mxfp8_rmsnorm_quantize(int fmt, const void* x_bf16, int64_t x_stride, const void* residual,
                                    int64_t residual_stride, int residual_is_f32, void* residual_out,
                                    const void* weight_bf16, float eps, const float* tensor_scale, int64_t M, int64_t K,
                                    uint8_t* q, uint8_t* scale, int scale_packed, void* y_bf16,
                                    mxfp8_stream_t stream) {
  mxfp8_status st = check_qfmt(fmt);
  if (st != MXFP8_OK || (st = check_blocks(fmt, 1, M, K, "norm")) != MXFP8_OK ||
      (st = check_tensor_scale(fmt, tensor_scale)) != MXFP8_OK)
    return st;
  if (K > mx::kNormMaxK || M > 0x7FFFFFFFll)
    return fail(MXFP8_ERR_UNSUPPORTED, "norm: K=%lld (at most %lld), M=%lld", (long long)K, (long long)mx::kNormMaxK,
                (long long)M);
  if (!(eps >= 0.f)) return fail(MXFP8_ERR_INVALID_ARG, "norm: eps must be a number >= 0");
  if (M == 0) return MXFP8_OK;
  if ((st = check_rows("x", x_bf16, x_stride, M, K, 2)) != MXFP8_OK) return st;
  if ((residual == nullptr) != (residual_out == nullptr))
    return fail(MXFP8_ERR_INVALID_ARG, "residual and residual_out go together");
  if (residual != nullptr &&
      (st = check_rows("residual", residual, residual_stride, M, K, residual_is_f32 ? 4 : 2)) != MXFP8_OK)
    return st;
  if (weight_bf16 == nullptr || q == nullptr || scale == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(residual_out, 16) || !aligned(weight_bf16, 16) || !aligned(q, 16) || !aligned(scale, 16) ||
      !aligned(y_bf16, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  const mx::NormProblem p{fmt,         x_bf16, x_stride, residual, residual_stride, residual_is_f32 != 0,
                          residual_out, weight_bf16, y_bf16, eps, tensor_scale, M, K, q, scale, scale_packed != 0};
  cudaError_t e = mx::launch_rmsnorm_quantize(p, as_stream(stream));
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "norm launch");
}

mxfp8_status mxfp8_silu_mul_quantize(int fmt, const void* gate_bf16, int64_t gate_stride, const void* up_bf16,
                                     int64_t up_stride, const float* tensor_scale, int64_t M, int64_t K, uint8_t* q,
                                     uint8_t* scale, int scale_packed, mxfp8_stream_t stream) {
  mxfp8_status st = check_qfmt(fmt);
  if (st != MXFP8_OK || (st = check_blocks(fmt, 1, M, K, "activation")) != MXFP8_OK ||
      (st = check_tensor_scale(fmt, tensor_scale)) != MXFP8_OK)
    return st;
  if (M == 0) return MXFP8_OK;
  if ((st = check_rows("gate", gate_bf16, gate_stride, M, K, 2)) != MXFP8_OK ||
      (st = check_rows("up", up_bf16, up_stride, M, K, 2)) != MXFP8_OK)
    return st;
  if (q == nullptr || scale == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(q, 16) || !aligned(scale, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  const mx::ActProblem p{fmt, gate_bf16, gate_stride, up_bf16, up_stride, tensor_scale, M, K, q, scale,
                         scale_packed != 0};
  cudaError_t e = mx::launch_silu_mul_quantize(p, as_stream(stream));
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "activation launch");
}

}  // extern "C"

namespace {

// The intermediates of a gated MLP block.
struct MlpLayout {
  int64_t aq, asf, h, cq, csf, part, part_bytes, total;
};

mxfp8_status mlp_layout(int fmt, int64_t M, int64_t K, int64_t F, MlpLayout* w) {
  mxfp8_status st = check_qfmt(fmt);
  if (st != MXFP8_OK || (st = check_blocks(fmt, 1, M, K, "MLP")) != MXFP8_OK ||
      (st = check_blocks(fmt, 1, M, F, "MLP")) != MXFP8_OK)
    return st;
  const int64_t per = fmt == MXFP8_QFMT_MXFP8 ? 1 : 2;
  int64_t p1 = 0, p2 = 0;
  if (fmt != MXFP8_QFMT_MXFP8 && M > 0) {
    if ((st = check_product(fmt, 1, M, 2 * F, K)) != MXFP8_OK || (st = check_product(fmt, 1, M, K, F)) != MXFP8_OK)
      return st;
    p1 = workspace_layout(fmt, 1, M, 2 * F, K, true, true, product_splits(1, M, 2 * F, K)).total;
    p2 = workspace_layout(fmt, 1, M, K, F, true, true, product_splits(1, M, K, F)).total;
  }
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  w->aq = take(M * K / per);
  w->asf = take(mx::sf_packed_bytes(1, M, fp4_scale_extent(fmt, K)));
  w->h = take(4 * M * F);
  w->cq = take(M * F / per);
  w->csf = take(mx::sf_packed_bytes(1, M, fp4_scale_extent(fmt, F)));
  w->part_bytes = p1 > p2 ? p1 : p2;
  w->part = take(w->part_bytes);
  w->total = at;
  return MXFP8_OK;
}

}  // namespace

extern "C" {

mxfp8_status mxfp8_gated_mlp_workspace_size(int fmt, int64_t M, int64_t K, int64_t F, size_t* bytes) {
  if (bytes == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null output pointer");
  MlpLayout w;
  mxfp8_status st = mlp_layout(fmt, M, K, F, &w);
  if (st == MXFP8_OK) *bytes = static_cast<size_t>(w.total);
  return st;
}

mxfp8_status mxfp8_gated_mlp(int fmt, const void* x_bf16, int64_t x_stride, const void* residual,
                             int64_t residual_stride, int residual_is_f32, void* residual_out,
                             const void* norm_weight_bf16, float eps, int64_t M, int64_t K, int64_t F,
                             const uint8_t* gate_up_packed, const uint8_t* gate_up_sf,
                             const float* gate_up_tensor_scale, const uint8_t* down_packed, const uint8_t* down_sf,
                             const float* down_tensor_scale, const float* a_tensor_scale, const float* c_tensor_scale,
                             void* out_bf16, void* workspace, size_t workspace_bytes, mxfp8_stream_t stream) {
  MlpLayout w;
  mxfp8_status st = mlp_layout(fmt, M, K, F, &w);
  if (st != MXFP8_OK) return st;
  // everything a later step would refuse is refused before the first launch
  const bool mx8 = fmt == MXFP8_QFMT_MXFP8;
  if (mx8 && (K % 128 != 0 || F % 128 != 0))
    return fail(MXFP8_ERR_UNSUPPORTED, "MLP: K=%lld and F=%lld must be multiples of 128 in MXFP8", (long long)K,
                (long long)F);
  if ((st = check_tensor_scale(fmt, gate_up_tensor_scale)) != MXFP8_OK ||
      (st = check_tensor_scale(fmt, down_tensor_scale)) != MXFP8_OK ||
      (st = check_tensor_scale(fmt, a_tensor_scale)) != MXFP8_OK ||
      (st = check_tensor_scale(fmt, c_tensor_scale)) != MXFP8_OK)
    return st;
  if (M == 0) return MXFP8_OK;
  if (mx8 && ((st = mx::check_block_count(1, 2 * F, K, "MLP")) != MXFP8_OK ||
              (st = mx::check_block_count(1, K, F, "MLP")) != MXFP8_OK))
    return st;
  if (gate_up_packed == nullptr || gate_up_sf == nullptr || down_packed == nullptr || down_sf == nullptr ||
      out_bf16 == nullptr)
    return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(gate_up_packed, 16) || !aligned(gate_up_sf, 16) || !aligned(down_packed, 16) || !aligned(down_sf, 16) ||
      !aligned(out_bf16, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  if (static_cast<int64_t>(workspace_bytes) < w.total)
    return fail(MXFP8_ERR_INVALID_ARG, "workspace has %zu bytes, needs %lld", workspace_bytes, (long long)w.total);
  if (workspace == nullptr || !aligned(workspace, 256))
    return fail(MXFP8_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t *aq = ws + w.aq, *asf = ws + w.asf, *h = ws + w.h, *cq = ws + w.cq, *csf = ws + w.csf;
  auto product = [&](const uint8_t* q, const uint8_t* sf, const float* g, int64_t N, int64_t Kp, const uint8_t* wp,
                     const uint8_t* wsf, const float* gw, void* out) {
    return mx8 ? mxfp8_gemm_packed(q, sf, 1, M, N, Kp, wp, wsf, nullptr, out, stream)
               : mxfp8_fp4_gemm_packed(fmt, q, sf, g, 1, M, N, Kp, wp, wsf, gw, nullptr, out,
                                       w.part_bytes > 0 ? ws + w.part : nullptr, static_cast<size_t>(w.part_bytes),
                                       stream);
  };
  st = mxfp8_rmsnorm_quantize(fmt, x_bf16, x_stride, residual, residual_stride, residual_is_f32, residual_out,
                              norm_weight_bf16, eps, a_tensor_scale, M, K, aq, asf, 1, nullptr, stream);
  if (st != MXFP8_OK) return st;
  st = product(aq, asf, a_tensor_scale, 2 * F, K, gate_up_packed, gate_up_sf, gate_up_tensor_scale, h);
  if (st != MXFP8_OK) return st;
  st = mxfp8_silu_mul_quantize(fmt, h, 2 * F, h + 2 * F, 2 * F, c_tensor_scale, M, F, cq, csf, 1, stream);
  if (st != MXFP8_OK) return st;
  return product(cq, csf, c_tensor_scale, K, F, down_packed, down_sf, down_tensor_scale, out_bf16);
}

}  // extern "C"
