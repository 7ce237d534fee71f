// mx_grouped.cuh - what the grouped product kernels share: instructions issued by
// one elected lane, the table of the groups, and the tiles.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_grouped.h"
#include "mx_layout.cuh"
#include "mx_ptx.cuh"

namespace mx {

constexpr int kGW_Rows = 128;  // weight rows (and, x on the M side, rows of x) per CTA
constexpr int kGBK = 128;      // bytes (elements) of K per row and stage: one block of fp8_128
constexpr int kGBox = 16;      // rows of x per copy of a tile that is not full

// ---------------------------------------------------------------- instructions issued by one elected lane
// as predicated instructions of a converged warp (see gemm_fp4.cu)
template <int CG>
__device__ __forceinline__ void mma_mxf8(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(elected)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

// Arrive on `bar` when all earlier MMAs of this lane are done: in both CTAs of a pair, or here.
template <int CG>
__device__ __forceinline__ void commit(uint32_t elected, uint64_t* bar) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3)), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(elected)
        : "memory");
}

// bar: shared-window address; on a pair the even CTA's.
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t elected, uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0,
                                         int c1, int c2) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];\n\t}" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(elected)
        : "memory");
}

__device__ __forceinline__ void expect_tx(uint32_t elected, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes), "r"(elected)
      : "memory");
}

template <int N>
__device__ __forceinline__ void set_registers_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_registers_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// mbar_wait without a call: the epilogue's sums would have to be saved around one.
__device__ __forceinline__ bool mbar_wait_inline(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > kWaitLimitNs) {
      atomicOr(&g_status, kStatusTimeout);
      *abort = 1;
      return false;
    }
  }
}

// ---------------------------------------------------------------- groups and tiles
struct GroupedArgs {
  const int* offsets;     // [groups + 1] on the device, or nullptr: every group has M rows
  int groups;
  int M;                  // rows of each group without offsets
  int R;                  // rows of x and out
  int N;
  int WT;                 // weight tiles of CG * 128 rows
  int KT;                 // stages of K
  int splits;             // K splits = cluster size (CG = 1)
  int offsets_ready;      // GroupedProblem::offsets_ready
  int w_fast;             // 1: weight tiles vary fastest within a group, 0: tiles of x
  const uint32_t* xs;     // scales of x: word (r, kt) at r * xs_row + kt * xs_kt holds the
  int64_t xs_row, xs_kt;  // four E8M0 bytes (MXFP8) or the fp32 (fp8_128) of 128 elements
  const void* ws;         // MXFP8: packed atoms; fp8_128: fp32 [groups][NB][KT]
  int RTW;                // weight row tiles of 128 (atoms), NB of fp8_128
  const __nv_bfloat16* bias;
  int64_t bias_stride;    // of a group: N, or 0 for one bias
  __nv_bfloat16* out;
  const __nv_bfloat16* x;  // quantised inside: bf16 [R, K]
  int K;
};

// The groups' first rows, row counts and the tiles before them.
struct GroupTable {
  int* start;
  int* count;
  int* before;  // [groups + 1]
};

bool grouped_maps(const GroupedProblem& p, int box_rows, CUtensorMap* mw, CUtensorMap* mx, CUtensorMap* mbox);
GroupedArgs grouped_args(const GroupedProblem& p, int cg, int splits);

// Fills the table from the offsets; all threads of the CTA.  Whatever the offsets
// hold, no row outside of x is touched: each is taken as at least 0 and the one
// before it, and at most R, so that groups never overlap and there are at most
// grouped_max_tiles tiles of up to tn rows.  A __syncthreads before and one after
// are the caller's; load_offsets comes first.
__device__ __forceinline__ void load_offsets(const GroupedArgs& a, const GroupTable& t, int nthreads) {
  for (int e = threadIdx.x; e <= a.groups; e += nthreads) t.before[e] = min(max(a.offsets[e], 0), a.R);
}
// One warp.  before[e + 1] is read before before[e] is overwritten.
template <int TN>
__device__ __forceinline__ void fill_table(const GroupedArgs& a, const GroupTable& t, int lane) {
  int sum = 0, top = 0;
  for (int e0 = 0; e0 < a.groups; e0 += 32) {
    const int e = e0 + lane;
    int start = e < a.groups ? t.before[e] : 0;
    const int next = e < a.groups ? t.before[e + 1] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, start, d);
      if (lane >= d) start = max(start, o);
    }
    start = max(start, top);
    const int count = e < a.groups ? max(next - start, 0) : 0;
    top = __shfl_sync(0xFFFFFFFFu, start + count, 31);
    const int mine = (count + TN - 1) / TN;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += o;
    }
    if (e < a.groups) {
      t.start[e] = start;
      t.count[e] = count;
      t.before[e] = sum + upto - mine;
    }
    sum += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  if (lane == 0) t.before[a.groups] = sum;
}

struct GroupTile {
  int e, wt;        // group, weight tile
  int row0, rows;   // first row of x, rows
  int width;        // rows rounded up to STEP
};

// Unit u: of group e, tiles (x tile, weight tile).  STEP = 0: tiles of TN rows, the
// rest in the last.  Else a group's rows are shared out evenly: n rows over T =
// ceil(n / TN) tiles of ceil(n / T), rounded up to STEP (TN / STEP is a power of
// two up to 8, for which every tile keeps a row).
template <int STEP, int TN>
__device__ __forceinline__ GroupTile tile_of(int u, const GroupedArgs& a, const GroupTable& t) {
  GroupTile r;
  int start, n, tiles, v;
  if (a.offsets == nullptr) {
    n = a.M;
    tiles = (n + TN - 1) / TN;
    const int per = tiles * a.WT;
    r.e = u / per;
    v = u - r.e * per;
    start = r.e * a.M;
  } else {
    const int q = u / a.WT;  // before[e] <= q < before[e + 1]
    int lo = 0, hi = a.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (t.before[mid] <= q)
        lo = mid;
      else
        hi = mid;
    }
    r.e = lo;
    n = t.count[lo];
    start = t.start[lo];
    tiles = t.before[lo + 1] - t.before[lo];
    v = u - t.before[lo] * a.WT;
  }
  int xt;
  if (a.w_fast) {
    xt = v / a.WT;
    r.wt = v - xt * a.WT;
  } else {
    r.wt = v / tiles;
    xt = v - r.wt * tiles;
  }
  const int share = STEP == 0 ? TN : ((n + tiles - 1) / tiles + (STEP ? STEP : 1) - 1) / (STEP ? STEP : 1) * STEP;
  r.row0 = start + xt * share;
  r.rows = min(share, n - xt * share);
  r.width = STEP == 0 ? TN : (r.rows + (STEP ? STEP : 1) - 1) / (STEP ? STEP : 1) * STEP;
  return r;
}
// (An empty group's tiles are none; the search above never ends on one, because
// before[e] <= q < before[e + 1] has a single solution, the last e with before[e] <= q.)

// All units of a call.
template <int TN>
__device__ __forceinline__ int unit_count(const GroupedArgs& a, const GroupTable& t) {
  return (a.offsets != nullptr ? t.before[a.groups] : a.groups * ((a.M + TN - 1) / TN)) * a.WT;
}

}  // namespace mx
