// route.cu - expert routing: which experts each token goes to, the order of the
// rows by expert, and each token's weighted sum afterwards.
//
// route: of token t the k largest logits, ties to the lowest expert; an expert whose
// logit is -inf or NaN is never chosen (a mask), so that a token may have fewer than
// k, or none: those slots get id -1, weight 0, position -1.  Weights: softmax over
// all experts (the never-chosen ones count 0) or sigmoid of the logit, in fp32; with
// renormalize divided by the sum of the token's chosen ones (in slot order); times
// scale.  Rows are sorted by expert, within an expert by token: a counting sort in
// which nothing depends on the order of atomics.  A CTA takes the same range of
// tokens in both kernels:
//   select: a warp a token, logits in registers, k rounds of a warp maximum (over
//     keys whose integer order is the logits' order); counts per CTA and expert;
//   place: a CTA adds up the counts of all CTAs before it, and ranks its tokens 64
//     at a time: a bit per token and expert, a row's rank is the number of lower bits
//     set.  No two tokens share a bit, so the atomic or is as good as a store.
// Up to 32 tokens (one CTA) both run in one launch.
//
// combine: out[t] = bf16( sum_j w[t, j] y[positions[t, j]] + add[t] ), the sum in
// fp32 in the order of the slots; slots without a row are left out.  Bound by
// reading y once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_grouped.h"
#include "mx_layout.cuh"
#include "mx_ptx.cuh"

namespace mx {

namespace {

constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr int GROUP = 64;          // tokens ranked at a time
constexpr int MAX_BLOCKS = 160;    // CTAs whose counts a CTA adds up, a multiple of 32

struct Args {
  const void* logits;
  int64_t stride;
  int64_t T;
  int64_t per_block;  // tokens of a CTA: up to GROUP, or a multiple of it
  int blocks;
  int E, k;
  int bf16, sigmoid, renormalize;
  float scale;
  int* ids;
  float* weights;
  int* offsets;
  int* rows;
  int* positions;
  int* counts;  // [E][MAX_BLOCKS]
};

__device__ __forceinline__ float load_logit(const Args& a, int64_t t, int e) {
  if (a.bf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.stride + e]);
  return static_cast<const float*>(a.logits)[t * a.stride + e];
}

// Integer whose unsigned order is the float's; 0 for -inf and NaN (never chosen).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 as +0: they tie
  if ((b & 0x7FFFFFFFu) > 0x7F800000u || b == 0xFF800000u) return 0u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// One token by one warp; key[i]: of expert 32 i + lane.  A lane keeps its largest
// (the first of equals); a round is a warp maximum, the lowest expert that has it,
// and a new largest in the lane it came from.
template <int NL>
__device__ __forceinline__ void select_token(const Args& a, int64_t t, int lane, uint32_t (&key)[NL], int* counts) {
  uint32_t best = 0;
  int at = 0;
  auto largest = [&]() {
    best = key[0];
    at = 0;
#pragma unroll
    for (int i = 1; i < NL; ++i) {
      if (key[i] > best) at = i;
      best = max(best, key[i]);
    }
  };
  largest();
  uint32_t most = __reduce_max_sync(0xFFFFFFFFu, best);
  const float top = key_value(most);
  float sum = 1.f;
  if (!a.sigmoid) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (key[i] != 0) sum += expf(key_value(key[i]) - top);
    sum = warp_sum(sum);
  }
  int my_id = -1;  // lane j keeps slot j
  uint32_t my_key = 0;
  for (int j = 0; j < a.k; ++j) {
    if (j > 0) most = __reduce_max_sync(0xFFFFFFFFu, best);
    if (most == 0) break;  // none is left
    const int id = __reduce_min_sync(0xFFFFFFFFu, best == most ? at * 32 + lane : 0x7FFFFFFF);
    if (lane == j) {
      my_id = id;
      my_key = most;
    }
    if ((id & 31) == lane) {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (i == at) key[i] = 0;
      largest();
      atomicAdd(&counts[id], 1);
    }
  }
  float my_w = 0.f;
  if (my_id >= 0) {
    const float v = key_value(my_key);
    my_w = a.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) / sum;
  }
  if (a.renormalize) {
    const float total = warp_sum(my_w);
    my_w = total > 0.f ? my_w / total : my_w;  // all zero: stay so
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = my_id;
    a.weights[t * a.k + lane] = my_w * a.scale;
  }
}

// The next token's logits are on their way while one is sorted.
template <int NL>
__device__ __forceinline__ void select_range(const Args& a, int64_t t0, int64_t t1, int* counts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float next[NL];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < NL; ++i) next[i] = t < t1 && i * 32 + lane < a.E ? load_logit(a, t, i * 32 + lane) : 0.f;
  };
  fetch(t0 + warp);
  for (int64_t t = t0 + warp; t < t1; t += warps) {
    uint32_t key[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) key[i] = i * 32 + lane < a.E ? order_key(next[i]) : 0u;
    fetch(t + warps);
    select_token<NL>(a, t, lane, key, counts);
  }
}

__device__ __forceinline__ void select_any(const Args& a, int64_t t0, int64_t t1, int* counts) {
  if (a.E <= 32)
    select_range<1>(a, t0, t1, counts);
  else if (a.E <= 64)
    select_range<2>(a, t0, t1, counts);
  else if (a.E <= 128)
    select_range<4>(a, t0, t1, counts);
  else if (a.E <= 256)
    select_range<8>(a, t0, t1, counts);
  else
    select_range<16>(a, t0, t1, counts);
}

// Rows and positions of tokens [t0, t1), whose experts are in a.ids; next[e]: the row
// of the first of them (shared; advanced).  A thread clears the words whose bits it has
// just counted: nobody else touches them between the two barriers around that.
__device__ __forceinline__ void place_range(const Args& a, int64_t t0, int64_t t1, int* next, uint32_t* mask) {
  for (int e = threadIdx.x; e < 2 * a.E; e += THREADS) mask[e] = 0;
  for (int64_t g0 = t0; g0 < t1; g0 += GROUP) {
    const int slots = static_cast<int>(min(static_cast<int64_t>(GROUP), t1 - g0)) * a.k;
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += THREADS) {
      const int e = a.ids[g0 * a.k + i], t = i / a.k;
      if (e >= 0) atomicOr(&mask[2 * e + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += THREADS) {
      const int e = a.ids[g0 * a.k + i], t = i / a.k;
      int pos = -1;
      if (e >= 0) {
        const uint32_t lo = mask[2 * e], hi = mask[2 * e + 1], below = (1u << (t & 31)) - 1u;
        pos = next[e] + (t < 32 ? __popc(lo & below) : __popc(lo) + __popc(hi & below));
        a.rows[pos] = static_cast<int>(g0 + t);
      }
      a.positions[g0 * a.k + i] = pos;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += THREADS) {
      next[e] += __popc(mask[2 * e]) + __popc(mask[2 * e + 1]);
      mask[2 * e] = mask[2 * e + 1] = 0;
    }
  }
}

// Exclusive sums of total[0 .. E) (E <= THREADS), thread e's in the return value;
// the whole sum in *all.
__device__ __forceinline__ int scan(int total, int* warp_sums, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = total;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += warp_sums[w];
    sum += warp_sums[w];
  }
  *all = sum;
  return before + upto - total;
}

// kOne: one CTA does everything; else the selection and its counts.
template <bool kOne>
__global__ void __launch_bounds__(THREADS) route_select_kernel(const Args a) {
  __shared__ int counts[kRouteMaxE];
  __shared__ uint32_t mask[2 * kRouteMaxE];
  __shared__ int warp_sums[WARPS];
  launch_dependents();
  const int64_t t0 = blockIdx.x * a.per_block, t1 = min(t0 + a.per_block, a.T);
  for (int e = threadIdx.x; e < a.E; e += THREADS) counts[e] = 0;
  __syncthreads();
  grid_dependency_wait();
  select_any(a, t0, t1, counts);
  __syncthreads();  // counts and (kOne) this CTA's ids
  if (!kOne) {
    for (int e = threadIdx.x; e < a.E; e += THREADS) a.counts[e * MAX_BLOCKS + blockIdx.x] = counts[e];
    return;
  }
  int all;
  const int e = threadIdx.x;
  const int first = scan(e < a.E ? counts[e] : 0, warp_sums, &all);
  __syncthreads();
  if (e < a.E) {
    counts[e] = first;
    a.offsets[e] = first;
  }
  if (e == 0) a.offsets[a.E] = all;
  for (int64_t i = all + threadIdx.x; i < a.T * a.k; i += THREADS) a.rows[i] = -1;
  __syncthreads();
  place_range(a, t0, t1, counts, mask);
}

__global__ void __launch_bounds__(THREADS) route_place_kernel(const Args a) {
  __shared__ int next[kRouteMaxE];
  __shared__ int totals[kRouteMaxE];
  __shared__ uint32_t mask[2 * kRouteMaxE];
  __shared__ int warp_sums[WARPS];
  launch_dependents();
  const int mine = static_cast<int>(blockIdx.x), lane = threadIdx.x & 31;
  grid_dependency_wait();
  // a warp an expert, a lane every 32nd CTA; four experts' counts in flight
  for (int e0 = (threadIdx.x >> 5) * 4; e0 < a.E; e0 += 4 * WARPS) {
    int c[4][MAX_BLOCKS / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < MAX_BLOCKS / 32; ++j)
        c[i][j] = e0 + i < a.E && 32 * j + lane < a.blocks ? a.counts[(e0 + i) * MAX_BLOCKS + 32 * j + lane] : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int total = 0, before = 0;
#pragma unroll
      for (int j = 0; j < MAX_BLOCKS / 32; ++j) {
        total += c[i][j];
        if (32 * j + lane < mine) before += c[i][j];
      }
      total = __reduce_add_sync(0xFFFFFFFFu, total);
      before = __reduce_add_sync(0xFFFFFFFFu, before);
      if (lane == 0 && e0 + i < a.E) {
        totals[e0 + i] = total;
        next[e0 + i] = before;
      }
    }
  }
  __syncthreads();
  const int e = threadIdx.x;
  const int total = e < a.E ? totals[e] : 0;
  int all;
  const int first = scan(total, warp_sums, &all);
  if (e < a.E) {
    next[e] += first;
    if (blockIdx.x == 0) a.offsets[e] = first;
  }
  if (blockIdx.x == 0 && e == 0) a.offsets[a.E] = all;
  for (int64_t i = all + blockIdx.x * THREADS + threadIdx.x; i < a.T * a.k; i += static_cast<int64_t>(a.blocks) * THREADS)
    a.rows[i] = -1;
  __syncthreads();
  const int64_t t0 = blockIdx.x * a.per_block;
  place_range(a, t0, min(t0 + a.per_block, a.T), next, mask);
}

// Tokens a CTA takes: all where a warp has one; else at most MAX_BLOCKS CTAs with up to
// GROUP each, or whole groups.  (2048 tokens, 64 experts, 32 CTAs 11.8 us, 128 8.9; 64
// tokens in one CTA and launch 8.1, 8 CTAs 6.7.  From 10241 tokens on whole groups, up to
// half of the CTAs: 64 experts, 10240 tokens 18.0, 10241 18.9, 16384 19.0, 30000 39.7.)
int64_t tokens_per_block(int64_t T) {
  if (T <= WARPS) return WARPS;
  const int64_t even = ceil_div(T, MAX_BLOCKS);
  return even <= GROUP ? ceil_div(even, 8) * 8 : ceil_div(even, GROUP) * GROUP;
}

struct CombineArgs {
  const __nv_bfloat16* y;
  const int* positions;
  const float* weights;
  const __nv_bfloat16* add;
  int64_t add_stride;
  int64_t T, R, N;
  int k;
  int64_t tasks;  // T * segs
  int segs;       // a task: up to 256 columns of a token, eight a lane
  __nv_bfloat16* out;
};

__device__ __forceinline__ void add_bf16x8(float (&acc)[8], const uint4 v, float w) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(__uint_as_float(r[i] << 16), w, acc[2 * i]);
    acc[2 * i + 1] = fmaf(__uint_as_float(r[i] & 0xFFFF0000u), w, acc[2 * i + 1]);
  }
}

constexpr int COMBINE_THREADS = 256;

// A warp a task; lane j holds slot j's row and weight, eight rows are in flight.
__global__ void __launch_bounds__(COMBINE_THREADS) combine_kernel(const CombineArgs a) {
  launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (COMBINE_THREADS / 32) + (threadIdx.x >> 5);
  if (task >= a.tasks) return;
  const int64_t t = task / a.segs;
  const int64_t c = (task - t * a.segs) * 256 + lane * 8;
  grid_dependency_wait();
  int pos = -1;
  float w = 0.f;
  if (lane < a.k) {
    pos = a.positions[t * a.k + lane];
    w = a.weights[t * a.k + lane];
    if (pos >= a.R) pos = -1;
  }
  float acc[8] = {};
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = __shfl_sync(0xFFFFFFFFu, pos, (j0 + j) & 31);
      if (j0 + j < a.k && p >= 0 && c < a.N) v[j] = *reinterpret_cast<const uint4*>(a.y + p * a.N + c);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = __shfl_sync(0xFFFFFFFFu, pos, (j0 + j) & 31);
      const float wj = __shfl_sync(0xFFFFFFFFu, w, (j0 + j) & 31);
      if (j0 + j < a.k && p >= 0 && c < a.N) add_bf16x8(acc, v[j], wj);
    }
  }
  if (c >= a.N) return;
  if (a.add != nullptr) add_bf16x8(acc, *reinterpret_cast<const uint4*>(a.add + t * a.add_stride + c), 1.f);
  *reinterpret_cast<uint4*>(a.out + t * a.N + c) = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                                             pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
}

cudaError_t launch(const void* fn, int64_t blocks, int threads, void** args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

int64_t route_count_bytes(int64_t T, int E) {
  const int64_t blocks = ceil_div(T, tokens_per_block(T > 0 ? T : 1));
  return blocks > 1 ? 4ll * MAX_BLOCKS * E : 0;
}

cudaError_t launch_route(const RouteProblem& p, cudaStream_t stream) {
  Args a;
  a.logits = p.logits;
  a.stride = p.stride;
  a.T = p.T;
  a.per_block = tokens_per_block(p.T);
  a.blocks = static_cast<int>(ceil_div(p.T, a.per_block));
  a.E = p.E;
  a.k = p.k;
  a.bf16 = p.bf16;
  a.sigmoid = p.sigmoid;
  a.renormalize = p.renormalize;
  a.scale = p.scale;
  a.ids = p.ids;
  a.weights = p.weights;
  a.offsets = p.offsets;
  a.rows = p.rows;
  a.positions = p.positions;
  a.counts = p.counts;
  void* args[] = {&a};
  if (a.blocks == 1)
    return launch(reinterpret_cast<const void*>(route_select_kernel<true>), 1, THREADS, args, stream);
  cudaError_t e = launch(reinterpret_cast<const void*>(route_select_kernel<false>), a.blocks, THREADS, args, stream);
  if (e != cudaSuccess) return e;
  return launch(reinterpret_cast<const void*>(route_place_kernel), a.blocks, THREADS, args, stream);
}

cudaError_t launch_combine(const CombineProblem& p, cudaStream_t stream) {
  CombineArgs a;
  a.y = static_cast<const __nv_bfloat16*>(p.y);
  a.positions = p.positions;
  a.weights = p.weights;
  a.add = static_cast<const __nv_bfloat16*>(p.add);
  a.add_stride = p.add_stride;
  a.T = p.T;
  a.R = p.R;
  a.N = p.N;
  a.k = p.k;
  a.segs = static_cast<int>(ceil_div(p.N, 256));
  a.tasks = p.T * a.segs;
  a.out = static_cast<__nv_bfloat16*>(p.out);
  void* args[] = {&a};
  return launch(reinterpret_cast<const void*>(combine_kernel), ceil_div(a.tasks, COMBINE_THREADS / 32), COMBINE_THREADS,
                args, stream);
}

}  // namespace mx
