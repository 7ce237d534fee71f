// api_grouped.cu - the C ABI of the block-128 FP8 layer, the products grouped by
// expert, the expert routing and the mixture-of-experts MLP (declared in
// include/mxfp8.h).  Host side only: argument checks (all before any launch),
// workspace carving and the choice of kernels.
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_api.h"
#include "mx_grouped.h"
#include "mx_kernels.h"
#include "mx_layout.cuh"

static_assert(MXFP8_GFMT_MXFP8 == mx::kG8MX && MXFP8_GFMT_FP8_128 == mx::kG8B128, "format codes");

namespace {

using mx::aligned;
using mx::ceil_div;
using mx::cuda_fail;
using mx::fail;
using mx::round_up;

typedef long long ll;

cudaStream_t as_stream(mxfp8_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int64_t kMaxRows = 1ll << 30;
constexpr int64_t kMaxExtent = 1ll << 27;

mxfp8_status check_gfmt(int fmt) {
  if (fmt != MXFP8_GFMT_MXFP8 && fmt != MXFP8_GFMT_FP8_128) return fail(MXFP8_ERR_INVALID_ARG, "format %d", fmt);
  return MXFP8_OK;
}

// Rows of E4M3 elements with their scales along K.
mxfp8_status check_rows_k(int fmt, int64_t R, int64_t K, const char* what) {
  if (R < 0 || K < 1) return fail(MXFP8_ERR_INVALID_ARG, "%s: rows=%lld K=%lld", what, (ll)R, (ll)K);
  if (fmt == MXFP8_GFMT_MXFP8 && K % 128 != 0)
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: K=%lld must be a multiple of 128 in MXFP8", what, (ll)K);
  if (K % 16 != 0) return fail(MXFP8_ERR_UNSUPPORTED, "%s: K=%lld must be a multiple of 16", what, (ll)K);
  if (R > kMaxRows || K > kMaxExtent || (R > 0 && ceil_div(K, 512) > (1ll << 33) / R))
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: rows=%lld K=%lld is too large; split the call", what, (ll)R, (ll)K);
  return MXFP8_OK;
}

mxfp8_status check_product(int fmt, int64_t E, int64_t R, int64_t N, int64_t K, bool ragged) {
  mxfp8_status st = check_gfmt(fmt);
  if (st != MXFP8_OK || (st = check_rows_k(fmt, R, K, "activations")) != MXFP8_OK) return st;
  if (E < 1 || N < 1) return fail(MXFP8_ERR_INVALID_ARG, "groups=%lld N=%lld", (ll)E, (ll)N);
  if (N % 8 != 0) return fail(MXFP8_ERR_UNSUPPORTED, "N=%lld: this library needs N %% 8 == 0", (ll)N);
  if (ragged && E > mx::kMaxGroups)
    return fail(MXFP8_ERR_UNSUPPORTED, "%lld groups: at most %d", (ll)E, mx::kMaxGroups);
  if (N > kMaxExtent || E > (1ll << 20)) return fail(MXFP8_ERR_UNSUPPORTED, "groups=%lld N=%lld is too large", (ll)E, (ll)N);
  if (fmt == MXFP8_GFMT_MXFP8 && (st = mx::check_block_count(E, N, K, "weights")) != MXFP8_OK) return st;
  // output tiles (128 rows x 16 columns at the least) are counted in 31 bits
  if (E * ceil_div(N, 128) > (1ll << 30) || (E + ceil_div(R, 16)) > (1ll << 30) / ceil_div(N, 128))
    return fail(MXFP8_ERR_UNSUPPORTED, "groups=%lld rows=%lld N=%lld has too many output tiles", (ll)E, (ll)R, (ll)N);
  return MXFP8_OK;
}

// Codes and scale words of x quantised inside a call: [R, K], then [ceil(K / 128)][R].
// Where many rows are picked from at most a quarter as many tokens, the tokens are
// quantised first, [T, K] and [T][ceil(K / 128)], and their codes picked (us, the whole
// call in one step and in two, MXFP8, 16 experts of 2048 x 4096: 16384 rows from 2048
// tokens 118 / 107, from 8192 118 / 120; 4096 rows from 512 42.7 / 41.2, from 2048 42.6 /
// 44.0; 2048 rows from 256 34.6 / 35.5).
struct XLayout {
  int64_t s, tq, ts, total;
};

bool picks_codes(int64_t R, int64_t K) { return R * K >= 1ll << 24; }

XLayout x_layout(int64_t R, int64_t K, bool ragged) {
  const int64_t most = ragged && picks_codes(R, K) ? R / 4 : 0, KT = ceil_div(K, 128);
  XLayout w;
  w.s = round_up(R * K, 256);
  w.tq = w.s + round_up(4 * R * KT, 256);
  w.ts = w.tq + round_up(most * K, 256);
  w.total = w.ts + round_up(4 * most * KT, 256);
  return w;
}

struct Product {
  int fmt;
  int64_t E, R, N, K;
  const void* x_bf16;  // [T, K], or null with x_q, x_scale
  int64_t T;
  const int* rows;
  const uint8_t* x_q;
  const void* x_scale;
  const int* offsets;
  const uint8_t* w;
  const void* ws;
  const void* bias;
  int64_t bias_stride;
  void* out;
};

// Scale words of a quantised x that a product wants K-block major: a warp reads those
// of 32 rows and one block at once, which row-major are in 32 cache lines.  On pairs in
// MXFP8 every one of four warps reads all of a tile's, and 16384 rows, 16 experts of
// 4096 x 4096 took 392 us instead of 210 (both with one set of scale warps;
// the call takes 185 now, this step in it).
int64_t turned_bytes(int fmt, int64_t E, int64_t R, int64_t N, int64_t K, bool ragged) {
  return fmt == MXFP8_GFMT_MXFP8 && mx::grouped_plan(fmt, E, R, N, K, ragged).cg == 2 ? round_up(4 * R * ceil_div(K, 128), 256) : 0;
}

// The checks of a product call, then its launches.
mxfp8_status run_product(const Product& p, void* workspace, size_t workspace_bytes, mxfp8_stream_t stream) {
  mxfp8_status st;
  const bool have_x = p.x_bf16 != nullptr, have_q = p.x_q != nullptr || p.x_scale != nullptr;
  if (have_x == have_q) return fail(MXFP8_ERR_INVALID_ARG, "pass exactly one of x_bf16 or (x_q, x_scale)");
  if (have_q && (p.x_q == nullptr || p.x_scale == nullptr))
    return fail(MXFP8_ERR_INVALID_ARG, "x_q and x_scale must both be given");
  if (have_q && p.rows != nullptr) return fail(MXFP8_ERR_INVALID_ARG, "rows go with bf16 x");
  if (p.w == nullptr || p.ws == nullptr || p.out == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(p.x_bf16, 16) || !aligned(p.x_q, 16) || !aligned(p.x_scale, 16) || !aligned(p.w, 16) ||
      !aligned(p.ws, 16) || !aligned(p.bias, 16) || !aligned(p.out, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  if (!aligned(p.rows, 4) || !aligned(p.offsets, 4))
    return fail(MXFP8_ERR_INVALID_ARG, "rows and offsets must be 4-byte aligned");
  const XLayout l = x_layout(p.R, p.K, p.offsets != nullptr);
  const int64_t turned = have_q ? turned_bytes(p.fmt, p.E, p.R, p.N, p.K, p.offsets != nullptr) : 0;
  const bool inside = have_x && p.fmt == MXFP8_GFMT_FP8_128 && p.rows == nullptr &&
                      mx::b128_quantizes_inside(p.offsets != nullptr, p.E, p.R);
  const int64_t need = inside ? 0 : (have_x ? l.total : turned);
  if (have_x) {
    if (p.T < 0 || p.T > kMaxRows || (p.rows == nullptr && p.T != p.R))
      return fail(MXFP8_ERR_INVALID_ARG, "x has %lld rows for %lld of the product", (ll)p.T, (ll)p.R);
  }
  if (need > 0) {
    if (static_cast<int64_t>(workspace_bytes) < need)
      return fail(MXFP8_ERR_INVALID_ARG, "workspace has %zu bytes, needs %lld", workspace_bytes, (ll)need);
    if (workspace == nullptr || !aligned(workspace, 256))
      return fail(MXFP8_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  }
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  const int64_t KT = ceil_div(p.K, 128);
  mx::GroupedProblem g;
  g.fmt = p.fmt;
  g.x = p.x_q;
  g.xs = p.x_scale;
  g.xs_row = KT;
  g.xs_kt = 1;
  g.w = p.w;
  g.ws = p.ws;
  g.bias = p.bias;
  g.bias_stride = p.bias_stride;
  g.out = p.out;
  g.offsets = p.offsets;
  g.E = p.E;
  g.R = p.R;
  g.N = p.N;
  g.K = p.K;
  if (inside) {
    g.x_bf16 = p.x_bf16;
  } else if (have_x) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const bool pick = p.rows != nullptr && p.T > 0 && p.T <= p.R / 4 && picks_codes(p.R, p.K);
    mx::QuantRowsProblem q{p.fmt, p.x_bf16, p.rows, p.T, p.R, p.K, ws, ws + l.s, 1, p.R, true};
    if (pick) q = mx::QuantRowsProblem{p.fmt, p.x_bf16, nullptr, p.T, p.T, p.K, ws + l.tq, ws + l.ts, KT, 1, true};
    cudaError_t e = mx::launch_quantize_rows(q, as_stream(stream));
    if (e == cudaSuccess && pick)
      e = mx::launch_gather_rows(ws + l.tq, ws + l.ts, p.rows, p.T, p.R, p.K, ws, ws + l.s, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "quantise launch");
    g.x = ws;
    g.xs = ws + l.s;
    g.xs_row = 1;
    g.xs_kt = p.R;
    g.offsets_ready = 1;
  } else if (turned > 0) {
    cudaError_t e = mx::launch_transpose_words(p.x_scale, p.R, KT, workspace, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "activation scale repack launch");
    g.xs = workspace;
    g.xs_row = 1;
    g.xs_kt = p.R;
    g.offsets_ready = 1;
  }
  const char* msg = "";
  cudaError_t e = mx::launch_gemm_grouped(g, mx::grouped_plan(p.fmt, p.E, p.R, p.N, p.K, p.offsets != nullptr), sms,
                                          as_stream(stream), &msg);
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, msg);
}

mxfp8_status check_strided(const char* what, const void* p, int64_t stride, int64_t M, int64_t K) {
  if (p == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned(p, 16) || (M > 1 && stride % 8 != 0))
    return fail(MXFP8_ERR_INVALID_ARG, "%s: rows must start on 16-byte boundaries (stride %lld)", what, (ll)stride);
  if (M > 1 && stride < K && stride != 0)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: row stride %lld is below %lld", what, (ll)stride, (ll)K);
  return MXFP8_OK;
}

mxfp8_status check_route(int64_t T, int64_t E, int64_t k, int scoring) {
  if (T < 0 || E < 1 || k < 1 || k > E)
    return fail(MXFP8_ERR_INVALID_ARG, "routing: tokens=%lld experts=%lld k=%lld", (ll)T, (ll)E, (ll)k);
  if (E > mx::kRouteMaxE || k > mx::kRouteMaxK)
    return fail(MXFP8_ERR_UNSUPPORTED, "routing: experts=%lld (at most %d), k=%lld (at most %d)", (ll)E, mx::kRouteMaxE,
                (ll)k, mx::kRouteMaxK);
  if (T > kMaxRows / k) return fail(MXFP8_ERR_UNSUPPORTED, "routing: %lld tokens are too many", (ll)T);
  if (scoring != MXFP8_ROUTE_SOFTMAX && scoring != MXFP8_ROUTE_SIGMOID)
    return fail(MXFP8_ERR_INVALID_ARG, "routing: scoring %d", scoring);
  return MXFP8_OK;
}

mxfp8_status check_logits(const void* logits, int64_t stride, int is_bf16, int64_t T, int64_t E) {
  if (logits == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(logits, is_bf16 ? 2 : 4)) return fail(MXFP8_ERR_INVALID_ARG, "logits must be aligned to their type");
  if (T > 1 && stride < E && stride != 0)
    return fail(MXFP8_ERR_INVALID_ARG, "logits: row stride %lld is below %lld", (ll)stride, (ll)E);
  return MXFP8_OK;
}

mxfp8_status check_combine(int64_t R, int64_t T, int64_t k, int64_t N) {
  if (R < 0 || T < 0 || k < 1 || N < 1)
    return fail(MXFP8_ERR_INVALID_ARG, "combine: rows=%lld tokens=%lld k=%lld N=%lld", (ll)R, (ll)T, (ll)k, (ll)N);
  if (N % 8 != 0) return fail(MXFP8_ERR_UNSUPPORTED, "combine: N=%lld must be a multiple of 8", (ll)N);
  if (k > mx::kRouteMaxK || R > kMaxRows || T > kMaxRows || N > kMaxExtent || (T > 0 && ceil_div(N, 256) > (1ll << 33) / T))
    return fail(MXFP8_ERR_UNSUPPORTED, "combine: rows=%lld tokens=%lld k=%lld N=%lld is too large", (ll)R, (ll)T, (ll)k, (ll)N);
  return MXFP8_OK;
}

// The intermediates of a mixture-of-experts MLP.
struct ExpertLayout {
  int64_t ids, weights, offsets, rows, positions, counts, xq, xs, h, cq, cs, total;
};

mxfp8_status expert_layout(int fmt, int64_t T, int64_t E, int64_t k, int64_t K, int64_t F, ExpertLayout* w) {
  mxfp8_status st = check_route(T, E, k, MXFP8_ROUTE_SOFTMAX);
  if (st != MXFP8_OK) return st;
  const int64_t R = T * k;
  if (F < 1 || F > kMaxExtent / 2) return fail(MXFP8_ERR_INVALID_ARG, "experts: F=%lld", (ll)F);
  if ((st = check_product(fmt, E, R, 2 * F, K, true)) != MXFP8_OK ||
      (st = check_product(fmt, E, R, K, F, true)) != MXFP8_OK || (st = check_combine(R, T, k, K)) != MXFP8_OK)
    return st;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  w->ids = take(4 * R);
  w->weights = take(4 * R);
  w->offsets = take(4 * (E + 1));
  w->rows = take(4 * R);
  w->positions = take(4 * R);
  w->counts = take(mx::route_count_bytes(T, static_cast<int>(E)));
  w->xq = take(R * K);
  w->xs = take(4 * R * ceil_div(K, 128));
  w->h = take(4 * R * F > 2 * R * K ? 4 * R * F : 2 * R * K);  // gate and up, then the down product
  w->cq = take(R * F);
  w->cs = take(4 * R * ceil_div(F, 128));
  w->total = at;
  return MXFP8_OK;
}

}  // namespace

extern "C" {

mxfp8_status mxfp8_b128_quantize(const void* x_bf16, int64_t rows, int64_t K, uint8_t* x_q, float* x_scale,
                                 mxfp8_stream_t stream) {
  mxfp8_status st = check_rows_k(MXFP8_GFMT_FP8_128, rows, K, "block-128 quantise");
  if (st != MXFP8_OK) return st;
  if (rows == 0) return MXFP8_OK;
  if (x_bf16 == nullptr || x_q == nullptr || x_scale == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(x_bf16, 16) || !aligned(x_q, 16) || !aligned(x_scale, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "x, codes and scales must be 16-byte aligned");
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  const mx::QuantRowsProblem q{mx::kG8B128, x_bf16, nullptr, rows, rows, K, x_q, x_scale, ceil_div(K, 128), 1, false};
  cudaError_t e = mx::launch_quantize_rows(q, as_stream(stream));
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "block-128 quantise launch");
}

mxfp8_status mxfp8_b128_quantize_weights(const void* w_bf16, int64_t B, int64_t N, int64_t K, uint8_t* w_q,
                                         float* w_scale, mxfp8_stream_t stream) {
  mxfp8_status st = check_rows_k(MXFP8_GFMT_FP8_128, N, K, "block-128 weights");
  if (st != MXFP8_OK) return st;
  if (B < 1 || N < 1) return fail(MXFP8_ERR_INVALID_ARG, "B=%lld N=%lld", (ll)B, (ll)N);
  if (B > (1ll << 20) || B * ceil_div(N, 128) > (1ll << 31) / ceil_div(K, 128) - 1)
    return fail(MXFP8_ERR_UNSUPPORTED, "B=%lld N=%lld K=%lld has too many blocks", (ll)B, (ll)N, (ll)K);
  if (w_bf16 == nullptr || w_q == nullptr || w_scale == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(w_bf16, 16) || !aligned(w_q, 16) || !aligned(w_scale, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "weights, codes and scales must be 16-byte aligned");
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  cudaError_t e = mx::launch_quantize_weights_b128(w_bf16, B, N, K, w_q, w_scale, as_stream(stream));
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "block-128 weight quantise launch");
}

mxfp8_status mxfp8_b128_silu_mul_quantize(const void* gate_bf16, int64_t gate_stride, const void* up_bf16,
                                          int64_t up_stride, int64_t M, int64_t K, uint8_t* q, float* scale,
                                          mxfp8_stream_t stream) {
  mxfp8_status st = check_rows_k(MXFP8_GFMT_FP8_128, M, K, "activation");
  if (st != MXFP8_OK) return st;
  if (M == 0) return MXFP8_OK;
  if ((st = check_strided("gate", gate_bf16, gate_stride, M, K)) != MXFP8_OK ||
      (st = check_strided("up", up_bf16, up_stride, M, K)) != MXFP8_OK)
    return st;
  if (q == nullptr || scale == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(q, 16) || !aligned(scale, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  const mx::ActRowsProblem p{mx::kG8B128, gate_bf16, gate_stride, up_bf16, up_stride, M, K, q, scale, ceil_div(K, 128), 1};
  cudaError_t e = mx::launch_silu_mul_rows(p, as_stream(stream));
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "activation launch");
}

mxfp8_status mxfp8_b128_workspace_size(int64_t B, int64_t M, int64_t N, int64_t K, int x_is_quantized, size_t* bytes) {
  if (bytes == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null output pointer");
  if (B < 1 || M < 0 || M > kMaxRows || B > kMaxRows)
    return fail(MXFP8_ERR_INVALID_ARG, "B=%lld M=%lld", (ll)B, (ll)M);
  mxfp8_status st = check_product(MXFP8_GFMT_FP8_128, B, B * M, N, K, false);
  if (st == MXFP8_OK)
    *bytes = x_is_quantized || mx::b128_quantizes_inside(false, B, B * M) ? 0 : static_cast<size_t>(x_layout(B * M, K, false).total);
  return st;
}

mxfp8_status mxfp8_b128_linear(const void* x_bf16, const uint8_t* x_q, const float* x_scale, int64_t B, int64_t M,
                               int64_t N, int64_t K, const uint8_t* w, const float* w_scale, const void* bias_bf16,
                               void* out_bf16, void* workspace, size_t workspace_bytes, mxfp8_stream_t stream) {
  if (B < 1 || M < 0 || M > kMaxRows || B > kMaxRows)
    return fail(MXFP8_ERR_INVALID_ARG, "B=%lld M=%lld", (ll)B, (ll)M);
  mxfp8_status st = check_product(MXFP8_GFMT_FP8_128, B, B * M, N, K, false);
  if (st != MXFP8_OK) return st;
  if (M == 0) return MXFP8_OK;
  const Product p{MXFP8_GFMT_FP8_128, B, B * M, N, K, x_bf16, B * M, nullptr, x_q, x_scale, nullptr, w, w_scale,
                  bias_bf16, 0, out_bf16};
  return run_product(p, workspace, workspace_bytes, stream);
}

mxfp8_status mxfp8_grouped_workspace_size(int fmt, int64_t E, int64_t R, int64_t N, int64_t K, int x_is_quantized,
                                          size_t* bytes) {
  if (bytes == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null output pointer");
  mxfp8_status st = check_product(fmt, E, R, N, K, true);
  if (st == MXFP8_OK)
    *bytes = static_cast<size_t>(R == 0 ? 0 : x_is_quantized ? turned_bytes(fmt, E, R, N, K, true) : x_layout(R, K, true).total);
  return st;
}

mxfp8_status mxfp8_grouped_linear(int fmt, const void* x_bf16, int64_t T, const int32_t* rows, const uint8_t* x_q,
                                  const void* x_scale, const int32_t* offsets, int64_t E, int64_t R, int64_t N,
                                  int64_t K, const uint8_t* w, const void* w_scale, const void* bias_bf16,
                                  void* out_bf16, void* workspace, size_t workspace_bytes, mxfp8_stream_t stream) {
  mxfp8_status st = check_product(fmt, E, R, N, K, true);
  if (st != MXFP8_OK) return st;
  if (R == 0) return MXFP8_OK;
  if (offsets == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null offsets");
  const Product p{fmt, E, R, N, K, x_bf16, T, rows, x_q, x_scale, offsets, w, w_scale, bias_bf16, N, out_bf16};
  return run_product(p, workspace, workspace_bytes, stream);
}

mxfp8_status mxfp8_route_workspace_size(int64_t T, int64_t E, int64_t k, size_t* bytes) {
  if (bytes == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null output pointer");
  mxfp8_status st = check_route(T, E, k, MXFP8_ROUTE_SOFTMAX);
  if (st == MXFP8_OK) *bytes = static_cast<size_t>(mx::route_count_bytes(T, static_cast<int>(E)));
  return st;
}

mxfp8_status mxfp8_route(const void* logits, int64_t logits_stride, int logits_are_bf16, int64_t T, int64_t E, int64_t k,
                         int scoring, int renormalize, float scale, int32_t* ids, float* weights, int32_t* offsets,
                         int32_t* rows, int32_t* positions, void* workspace, size_t workspace_bytes,
                         mxfp8_stream_t stream) {
  mxfp8_status st = check_route(T, E, k, scoring);
  if (st != MXFP8_OK) return st;
  if (offsets == nullptr || !aligned(offsets, 4)) return fail(MXFP8_ERR_INVALID_ARG, "offsets: null or misaligned");
  int sms = 0;
  if (T == 0) {  // every expert has no row
    if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
    cudaError_t e = cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * 4, as_stream(stream));
    return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "offsets");
  }
  if ((st = check_logits(logits, logits_stride, logits_are_bf16, T, E)) != MXFP8_OK) return st;
  if (ids == nullptr || weights == nullptr || rows == nullptr || positions == nullptr)
    return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(rows, 4) || !aligned(positions, 4))
    return fail(MXFP8_ERR_INVALID_ARG, "outputs must be 4-byte aligned");
  const int64_t need = mx::route_count_bytes(T, static_cast<int>(E));
  if (static_cast<int64_t>(workspace_bytes) < need)
    return fail(MXFP8_ERR_INVALID_ARG, "workspace has %zu bytes, needs %lld", workspace_bytes, (ll)need);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 256)))
    return fail(MXFP8_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  const mx::RouteProblem p{logits, logits_stride, logits_are_bf16 != 0, T, static_cast<int>(E), static_cast<int>(k),
                           scoring == MXFP8_ROUTE_SIGMOID, renormalize != 0, scale, ids, weights, offsets, rows, positions,
                           static_cast<int*>(workspace)};
  cudaError_t e = mx::launch_route(p, as_stream(stream));
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "routing launch");
}

mxfp8_status mxfp8_combine(const void* y_bf16, int64_t R, const int32_t* positions, const float* weights, int64_t T,
                           int64_t k, int64_t N, const void* add_bf16, int64_t add_stride, void* out_bf16,
                           mxfp8_stream_t stream) {
  mxfp8_status st = check_combine(R, T, k, N);
  if (st != MXFP8_OK) return st;
  if (T == 0) return MXFP8_OK;
  if ((R > 0 && y_bf16 == nullptr) || positions == nullptr || weights == nullptr || out_bf16 == nullptr)
    return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(y_bf16, 16) || !aligned(out_bf16, 16) || !aligned(positions, 4) || !aligned(weights, 4))
    return fail(MXFP8_ERR_INVALID_ARG, "y and out must be 16-byte aligned, positions and weights 4-byte");
  if (add_bf16 != nullptr && (st = check_strided("add", add_bf16, add_stride, T, N)) != MXFP8_OK) return st;
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  const mx::CombineProblem p{y_bf16, positions, weights, add_bf16, add_stride, T, R, N, static_cast<int>(k), out_bf16};
  cudaError_t e = mx::launch_combine(p, as_stream(stream));
  return e == cudaSuccess ? MXFP8_OK : cuda_fail(e, "combine launch");
}

mxfp8_status mxfp8_expert_mlp_workspace_size(int fmt, int64_t T, int64_t E, int64_t k, int64_t K, int64_t F,
                                             size_t* bytes) {
  if (bytes == nullptr) return fail(MXFP8_ERR_INVALID_ARG, "null output pointer");
  ExpertLayout w = {};
  mxfp8_status st = expert_layout(fmt, T, E, k, K, F, &w);
  if (st == MXFP8_OK) *bytes = static_cast<size_t>(w.total);
  return st;
}

mxfp8_status mxfp8_expert_mlp(int fmt, const void* x_bf16, int64_t T, int64_t K, const void* logits,
                              int64_t logits_stride, int logits_are_bf16, int64_t E, int64_t k, int scoring,
                              int renormalize, float scale, int64_t F, const uint8_t* gate_up, const void* gate_up_scale,
                              const uint8_t* down, const void* down_scale, const void* add_bf16, int64_t add_stride,
                              void* out_bf16, void* workspace, size_t workspace_bytes, mxfp8_stream_t stream) {
  ExpertLayout w = {};
  mxfp8_status st = check_route(T, E, k, scoring);
  if (st != MXFP8_OK || (st = expert_layout(fmt, T, E, k, K, F, &w)) != MXFP8_OK) return st;
  // everything a later step would refuse is refused before the first launch
  if (T == 0) return MXFP8_OK;
  if (x_bf16 == nullptr || gate_up == nullptr || gate_up_scale == nullptr || down == nullptr || down_scale == nullptr ||
      out_bf16 == nullptr)
    return fail(MXFP8_ERR_INVALID_ARG, "null pointer");
  if (!aligned(x_bf16, 16) || !aligned(gate_up, 16) || !aligned(gate_up_scale, 16) || !aligned(down, 16) ||
      !aligned(down_scale, 16) || !aligned(out_bf16, 16))
    return fail(MXFP8_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  if ((st = check_logits(logits, logits_stride, logits_are_bf16, T, E)) != MXFP8_OK) return st;
  if (add_bf16 != nullptr && (st = check_strided("add", add_bf16, add_stride, T, K)) != MXFP8_OK) return st;
  if (static_cast<int64_t>(workspace_bytes) < w.total)
    return fail(MXFP8_ERR_INVALID_ARG, "workspace has %zu bytes, needs %lld", workspace_bytes, (ll)w.total);
  if (workspace == nullptr || !aligned(workspace, 256))
    return fail(MXFP8_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  int sms = 0;
  if ((st = mx::current_device(&sms)) != MXFP8_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t R = T * k;
  int32_t *offsets = reinterpret_cast<int32_t*>(ws + w.offsets), *rows = reinterpret_cast<int32_t*>(ws + w.rows),
          *positions = reinterpret_cast<int32_t*>(ws + w.positions);
  float* weights = reinterpret_cast<float*>(ws + w.weights);
  uint8_t *xq = ws + w.xq, *h = ws + w.h, *cq = ws + w.cq;
  st = mxfp8_route(logits, logits_stride, logits_are_bf16, T, E, k, scoring, renormalize, scale,
                   reinterpret_cast<int32_t*>(ws + w.ids), weights, offsets, rows, positions, ws + w.counts,
                   static_cast<size_t>(mx::route_count_bytes(T, static_cast<int>(E))), stream);
  if (st != MXFP8_OK) return st;
  const mx::QuantRowsProblem q{fmt, x_bf16, nullptr, T, R, K, xq, ws + w.xs, 1, R, true, positions, static_cast<int>(k)};
  cudaError_t e = mx::launch_quantize_rows(q, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "quantise launch");
  const char* msg = "";
  mx::GroupedProblem g;
  g.fmt = fmt;
  g.x = xq;
  g.xs = ws + w.xs;
  g.xs_row = 1;
  g.xs_kt = R;
  g.w = gate_up;
  g.ws = gate_up_scale;
  g.bias = nullptr;
  g.bias_stride = 0;
  g.out = h;
  g.offsets = offsets;
  g.offsets_ready = 1;
  g.E = E;
  g.R = R;
  g.N = 2 * F;
  g.K = K;
  if ((e = mx::launch_gemm_grouped(g, mx::grouped_plan(fmt, E, R, 2 * F, K, true), sms, as_stream(stream), &msg)) !=
      cudaSuccess)
    return cuda_fail(e, msg);
  const mx::ActRowsProblem c{fmt, h, 2 * F, h + 2 * F, 2 * F, R, F, cq, ws + w.cs, 1, R};
  e = mx::launch_silu_mul_rows(c, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "activation launch");
  g.x = cq;
  g.xs = ws + w.cs;
  g.w = down;
  g.ws = down_scale;
  g.out = h;
  g.N = K;
  g.K = F;
  if ((e = mx::launch_gemm_grouped(g, mx::grouped_plan(fmt, E, R, K, F, true), sms, as_stream(stream), &msg)) !=
      cudaSuccess)
    return cuda_fail(e, msg);
  return mxfp8_combine(h, R, positions, weights, T, k, K, add_bf16, add_stride, out_bf16, stream);
}

}  // extern "C"
