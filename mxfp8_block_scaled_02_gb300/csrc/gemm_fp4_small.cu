// gemm_fp4_small.cu - the 4-bit product for few tokens or few output tiles:
//   out[b, m, n] = bf16( g_x g_w sum_k (x sx)[b, m, k] (w sw)[b, n, k] + bias[n] ).
//
// Bound by reading the weights once, and at decode sizes by the chain launch ->
// weights -> MMA -> reduction -> store.  So the weights are the MMA's M side
// (128 rows per CTA) and the tokens its N side (16, 32, 64 or 128 a CTA), no MMA
// row is padding, and K is split over a cluster of S CTAs so that every SM
// streams from the start: each holds a ring of 128-row x 128-byte weight tiles
// in flight before the tokens arrive (waited for with griddepcontrol.wait, like
// the bias and the tensor scales: any of them may be the previous kernel's output;
// the weights and their block scales may not).
// Codes and scale atoms of both operands come by TMA, the atoms go to tensor
// memory by tcgen05.cp in the MMA warp's own order.  A few bf16 tokens can
// also be quantised here (kQuant): six warps load the CTA's K range and write
// codes and scales where TMA would have put them, the bytes of the quantise
// call, which saves a launch and a workspace.
//
// The S fp32 partials meet in distributed shared memory, by stores that
// count on an mbarrier of the CTA they go to.  (With a releasing cluster barrier,
// and every mbarrier made by one thread, N = K = 4096, M = 1 took 4.0 us instead
// of 3.65; as bulk copies of a warp's partials, M = 128 9.2 instead of 7.1.)  CTA
// r owns weight rows [r 128/S, (r+1) 128/S) and adds the partials in the order
// 0..S-1, so the result is the same on every call; with S = 1 the epilogue stores
// straight from tensor memory.  With more tiles than SMs two CTAs share an SM
// (kTwo).
//
// Measured in a CUDA graph (us, MXFP4 / NVFP4): N = K = 4096, M = 1 3.6 / 3.7
// (bf16 x 3.8), 16 3.7 / 3.9, 64 5.2 / 5.3, 128 7.1 / 7.2; weights from HBM, N =
// 14336, K = 4096, M = 16 7.2 / 7.5 (31 MB, 4.3 TB/s: ~3 us of chain, then the
// stream), N = 28672, K = 4096 10.9 / 11.5 (62 MB, 5.7 TB/s).  On CTA pairs M = 1
// takes 8.5, 13 and 21.
//
// Warps: 0 weight TMA, 1 tensor-memory allocation and MMA issue, 2 token TMA
// (kQuant: 2..7 quantise the tokens), 4..7 epilogue; all eight reduce.  Every
// wait is bounded and the cluster barrier (at the start: the CTAs' mbarriers
// exist) is reached on every path.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_fp4.cuh"
#include "mx_kernels.h"
#include "mx_layout.cuh"
#include "mx_ptx.cuh"

namespace mx {

namespace {

constexpr int ROWS = 128;   // weight rows per CTA
constexpr int BKB = 128;    // bytes of K per row and stage
constexpr int BK = 2 * BKB;
constexpr int MMA_K = 64;
constexpr int THREADS = 256;
constexpr int W_BYTES = ROWS * BKB;

// kTwo: two CTAs an SM, each with a whole tile (no K split, so nothing received)
template <int FMT, int NTOK, bool kTwo>
struct Cfg {
  static constexpr int SMEM_MAX = kTwo ? 115712 : 232448;
  static constexpr int ATOMS = FMT == kQNV4 ? 4 : 2;
  static constexpr int SF_BYTES = ATOMS * kAtomBytes;  // scales of one operand and stage
  static constexpr int X_BYTES = NTOK * BKB;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES + 2 * SF_BYTES;
  static constexpr int RECV_BYTES = kTwo ? 0 : NTOK * ROWS * 4;  // [S][NTOK][ROWS / S] fp32
  static constexpr int FIT = (SMEM_MAX - 1024 - 512 - RECV_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = FIT < 12 ? FIT : 12;
  static constexpr int OFF_W = 0;
  static constexpr int OFF_X = OFF_W + STAGES * W_BYTES;
  static constexpr int OFF_SFW = OFF_X + STAGES * X_BYTES;
  static constexpr int OFF_SFX = OFF_SFW + STAGES * SF_BYTES;
  static constexpr int OFF_RECV = OFF_SFX + STAGES * SF_BYTES;
  static constexpr int OFF_BAR = OFF_RECV + RECV_BYTES;
  static constexpr int OFF_MISC = OFF_BAR + (3 * STAGES + 2) * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= SMEM_MAX && STAGES >= 3, "shared memory");
  // tensor memory: accumulator, then two scale slots (weight and token atoms)
  static constexpr int SLOT_COLS = 8 * ATOMS;
  static constexpr int T_SF = NTOK < 32 ? 32 : NTOK;
  static constexpr int T_END = T_SF + 2 * SLOT_COLS;
  static constexpr int TMEM_COLS = T_END <= 64 ? 64 : (T_END <= 128 ? 128 : 256);
  static_assert(T_END <= 256, "tensor memory");
};

template <int FMT>
__device__ __forceinline__ void mma_fp4(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (FMT == kQMX4)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], "
        "p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(elected)
        : "memory");
}

__device__ __forceinline__ void cp_sf(uint32_t elected, uint32_t taddr, uint64_t desc) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(desc), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void commit_elected(uint32_t elected, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}

__device__ __forceinline__ void tma_load_elected(uint32_t elected, uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                                 int c0, int c1, int c2) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];\n\t}" ::"r"(dst),
      "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void expect_tx_elected(uint32_t elected, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(elected)
      : "memory");
}

constexpr int QUANT_WARPS = 6;
constexpr int QUANT_MAX_M = 8;
constexpr int QUANT_AHEAD = 4;  // loads ahead, in tasks of two rows and a stage

struct Args {
  const __nv_bfloat16* x;  // kQuant: bf16 [M, K]
  int K;
  const __nv_bfloat16* bias;
  const float* gx;
  const float* gw;
  __nv_bfloat16* out;
  int M, N;
  int RTW, TT;     // weight row tiles, token tiles
  int KT;          // stages of K
  int last_steps;  // MMA steps of the last one
  int splits;      // cluster size S
};

template <int FMT, int NTOK, bool kQuant, bool kTwo>
__global__ void __launch_bounds__(THREADS, kTwo ? 2 : 1)
    gemm_fp4_small_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                          const __grid_constant__ CUtensorMap tmSFW, const __grid_constant__ CUtensorMap tmSFX,
                          const Args a) {
  using C = Cfg<FMT, NTOK, kTwo>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full_w = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full_x = full_w + C::STAGES;
  uint64_t* empty = full_x + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* received = acc_full + 1;  // the partials of the rows this CTA owns
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  // cluster = ((batch * TT) + token tile) * RTW + weight tile
  const int cluster = static_cast<int>(blockIdx.x) / a.splits;
  const int tile = cluster % a.RTW;
  const int tt = cluster / a.RTW % a.TT;
  const int b = cluster / a.RTW / a.TT;
  const int m0 = tt * NTOK;
  const int M = min(NTOK, a.M - m0);  // rows of this tile
  const int kt0 = rank * a.KT / a.splits;
  const int nk = (rank + 1) * a.KT / a.splits - kt0;  // >= 1: splits <= KT
  const uint32_t base = smem_u32(smem);

  if (warp == 0) {
    for (int i = lane; i < 3 * C::STAGES + 2; i += 32) mbar_init(&full_w[i], 1);
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
    __syncwarp();
    // S partials of 128 / S rows, in chunks of 16 tokens
    if (lane == 0 && a.splits > 1) mbar_arrive_expect_tx(received, static_cast<uint32_t>((M + 15) / 16 * 16 * ROWS * 4));
  }
  const uint32_t elected = elect_one();
  auto load_w = [&](int i, int st) {
    const uint32_t bar = smem_u32(&full_w[st]);
    expect_tx_elected(elected, bar, W_BYTES + C::SF_BYTES);
    tma_load_elected(elected, base + C::OFF_W + st * W_BYTES, &tmW, bar, (kt0 + i) * BKB, tile * ROWS, b);
    tma_load_elected(elected, base + C::OFF_SFW + st * C::SF_BYTES, &tmSFW, bar, tile * (kAtomBytes / 4),
                     (kt0 + i) * C::ATOMS, b);
  };
  const int first = nk < C::STAGES ? nk : C::STAGES;
  if (warp == 0) {
    // the first ring round needs nothing but the barriers this warp has made
    __syncwarp();
    for (int i = 0; i < first; ++i) load_w(i, i);
    launch_dependents();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (a.splits > 1) cluster_arrive_relaxed();  // this CTA's barriers exist
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  // the output row this thread finishes, its bias and the tensor scales
  const int per = ROWS / a.splits;
  const int my_n = a.splits == 1 ? tile * ROWS + (warp & 3) * 32 + lane
                                 : tile * ROWS + rank * per + static_cast<int>(threadIdx.x) % per;
  float bias_n = 0.f, alpha = 1.f;
  __nv_bfloat16* out = a.out + (static_cast<int64_t>(b) * a.M + m0) * a.N;

  if (warp == 0) {
    // ------------------------------------------------ weight producer, later rounds
    int st = 0, issued = first;
    uint32_t ph = 0;
    for (int i = first; i < nk; ++i) {
      if (!mbar_wait_warp(&empty[st], ph, abort_flag)) break;
      load_w(i, st);
      ++issued;
      if (++st == C::STAGES) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (*abort_flag) {  // leave with no copy in flight
      for (int s = 0; s < C::STAGES && s < issued; ++s)
        mbar_wait(&full_w[s], static_cast<uint32_t>(((issued - 1 - s) / C::STAGES) & 1), nullptr);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(NTOK >> 3) << 17) |
                               ((FMT == kQMX4 ? 1u : 0u) << 23) | (static_cast<uint32_t>(ROWS >> 4) << 24);
    const uint64_t wd0 = sdesc_kmajor_sw128(base + C::OFF_W), xd0 = sdesc_kmajor_sw128(base + C::OFF_X);
    const uint64_t sw0 = sdesc_sf(base + C::OFF_SFW), sx0 = sdesc_sf(base + C::OFF_SFX);
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = 0; i < nk; ++i) {
      if (!mbar_wait_warp(&full_w[st], ph, abort_flag) || !mbar_wait_warp(&full_x[st], ph, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t t_sfw = tmem + C::T_SF + (i & 1) * C::SLOT_COLS;
      const uint32_t t_sfx = t_sfw + 4 * C::ATOMS;
#pragma unroll
      for (int j = 0; j < C::ATOMS; ++j) {
        cp_sf(elected, t_sfw + 4 * j, sw0 + static_cast<uint32_t>((st * C::SF_BYTES + j * kAtomBytes) >> 4));
        cp_sf(elected, t_sfx + 4 * j, sx0 + static_cast<uint32_t>((st * C::SF_BYTES + j * kAtomBytes) >> 4));
      }
      const uint64_t wd = wd0 + static_cast<uint32_t>(st * (W_BYTES >> 4));
      const uint64_t xd = xd0 + static_cast<uint32_t>(st * (C::X_BYTES >> 4));
      const int steps = kt0 + i == a.KT - 1 ? a.last_steps : BK / MMA_K;
#pragma unroll
      for (int kk = 0; kk < BK / MMA_K; ++kk) {
        const int j = FMT == kQNV4 ? kk : kk >> 1;
        const uint32_t id = FMT == kQNV4 ? 0u : static_cast<uint32_t>(kk & 1) * 2u;
        mma_fp4<FMT>(kk < steps ? elected : 0u, tmem, wd + 2 * kk, xd + 2 * kk, idesc_with_sf_id(idesc, id, id),
                     t_sfw + 4 * j, t_sfx + 4 * j, (i | kk) != 0);
      }
      commit_elected(elected, &empty[st]);
      if (++st == C::STAGES) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (ok)
      commit_elected(elected, acc_full);
    else
      __nanosleep(200000);  // let issued tensor-core work retire
    __syncwarp();
  } else if (!kQuant && warp == 2) {
    // ------------------------------------------------ token producer
    grid_dependency_wait();
    int st = 0, issued = 0;
    uint32_t ph = 1;  // the first round's slots are free
    for (int i = 0; i < nk; ++i) {
      if (i >= C::STAGES && !mbar_wait_warp(&empty[st], ph, abort_flag)) break;
      const uint32_t bar = smem_u32(&full_x[st]);
      expect_tx_elected(elected, bar, C::X_BYTES + C::SF_BYTES);
      tma_load_elected(elected, base + C::OFF_X + st * C::X_BYTES, &tmX, bar, (kt0 + i) * BKB, m0, b);
      tma_load_elected(elected, base + C::OFF_SFX + st * C::SF_BYTES, &tmSFX, bar, tt * (kAtomBytes / 4),
                       (kt0 + i) * C::ATOMS, b);
      ++issued;
      if (++st == C::STAGES) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (*abort_flag) {
      for (int s = 0; s < C::STAGES && s < issued; ++s)
        mbar_wait(&full_x[s], static_cast<uint32_t>(((issued - 1 - s) / C::STAGES) & 1), nullptr);
    }
    __syncwarp();
  }
  if (kQuant && warp >= 2) {
    // ------------------------------------------------ token quantiser
    // QW warps take every QW-th stage; a task is two rows of it, 16 elements a
    // lane.  Task n of the warp: stage warp - 2 + QW (n / T), rows 2 (n % T) and
    // the one after, T = ceil(M / 2).  QW is at most the ring's length: a warp
    // that waits for stage i's slot has seen stage i - QW - STAGES consumed, and
    // the wait's parity is only right if that covers i - 2 STAGES.
    constexpr int QW = C::STAGES < QUANT_WARPS ? C::STAGES : QUANT_WARPS;
    grid_dependency_wait();
    const TensorScale ts = tensor_scale(FMT == kQNV4 && a.gx != nullptr ? *a.gx : 1.f);
    constexpr int kLanes = q_block(FMT) / 16;
    const int j = lane & 15, T = (a.M + 1) >> 1;
    const int ntasks = warp - 2 < QW ? (nk - (warp - 2) + QW - 1) / QW * T : 0;  // <= 0: none
    int lt = 0, li = warp - 2;  // task the next load belongs to
    auto load = [&](uint4 (&v)[2]) {
      const int r = 2 * lt + (lane >> 4), k = (kt0 + li) * BK + 16 * j;
      const bool valid = li < nk && r < a.M && k < a.K;
      const uint4* src = reinterpret_cast<const uint4*>(a.x + (valid ? static_cast<int64_t>(r) * a.K + k : 0));
      v[0] = valid ? src[0] : make_uint4(0, 0, 0, 0);
      v[1] = valid ? src[1] : make_uint4(0, 0, 0, 0);
      if (++lt == T) {
        lt = 0;
        li += QW;
      }
    };
    uint4 buf[QUANT_AHEAD][2];
#pragma unroll
    for (int d = 0; d < QUANT_AHEAD; ++d) load(buf[d]);
    int t = 0, i = warp - 2;
    bool ok = true;
    for (int n0 = 0; ok && n0 < ntasks; n0 += QUANT_AHEAD) {
#pragma unroll
      for (int d = 0; d < QUANT_AHEAD; ++d) {
        if (!ok || n0 + d >= ntasks) break;
        const int st = i % C::STAGES;
        if (t == 0 && i >= C::STAGES &&
            !mbar_wait_warp(&empty[st], static_cast<uint32_t>((i / C::STAGES - 1) & 1), abort_flag)) {
          ok = false;
          break;
        }
        const int r = 2 * t + (lane >> 4);
        const uint32_t w[8] = {buf[d][0].x, buf[d][0].y, buf[d][0].z, buf[d][0].w,
                               buf[d][1].x, buf[d][1].y, buf[d][1].z, buf[d][1].w};
        float f[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[2 * e] = __uint_as_float(w[e] << 16);
          f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
        load(buf[d]);
        uint32_t codes[4];
        uint32_t word = quantize_lane16<FMT>(f, ts, codes);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, kLanes) << 8;
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * kLanes) << 16;
        if (r < a.M) {
          // 128-byte swizzle: 16-byte piece q of row r sits at q ^ (r % 8)
          *reinterpret_cast<uint2*>(smem + C::OFF_X + st * C::X_BYTES + r * BKB + (((j >> 1) ^ (r & 7)) << 4) +
                                    (j & 1) * 8) = make_uint2(codes[0], codes[1]);
          if (j % (4 * kLanes) == 0)
            *reinterpret_cast<uint32_t*>(smem + C::OFF_SFX + st * C::SF_BYTES + j / (4 * kLanes) * kAtomBytes + r * 16) =
                word;
        }
        if (++t == T) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full_x[st]);
          t = 0;
          i += QW;
        }
      }
    }
    __syncwarp();
  }
  if (warp >= 4 || a.splits > 1) {
    // these, and the output's memory, may belong to the kernels before
    grid_dependency_wait();
    if (a.bias != nullptr && my_n < a.N) bias_n = __bfloat162float(a.bias[my_n]);
    if (a.gw != nullptr) alpha = *a.gw;
    if (a.gx != nullptr) alpha *= *a.gx;
  }
  if (a.splits > 1) cluster_wait();  // the other CTAs' barriers do
  if (warp >= 4 && mbar_wait_warp(acc_full, 0, abort_flag)) {
    // ------------------------------------------------ epilogue: lane = weight row
    tc_fence_after();
    const uint32_t lrow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int wrow = (warp & 3) * 32 + lane;
    const int owner = wrow / per;
    uint32_t dst = 0, bar = 0;
    if (a.splits > 1) {
      dst = map_shared_rank(base + C::OFF_RECV, static_cast<uint32_t>(owner)) +
            static_cast<uint32_t>(((rank * NTOK) * per + wrow - owner * per) * 4);
      bar = map_shared_rank(smem_u32(received), static_cast<uint32_t>(owner));
    }
    for (int c = 0; c < M; c += 16) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(lrow + c, r);
      tmem_ld_wait();
      if (a.splits == 1) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < M && my_n < a.N)
            out[static_cast<int64_t>(c + j) * a.N + my_n] =
                __float2bfloat16_rn(fmaf(__uint_as_float(r[j]), alpha, bias_n));
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) st_async_cluster_u32(dst + static_cast<uint32_t>((c + j) * per * 4), r[j], bar);
      }
    }
  }

  // Every partial of this CTA's rows has come, and none may come after it leaves
  // (each warp waits, whether or not it goes on).
  if (a.splits > 1 && mbar_wait_warp(received, 0, nullptr) && !*abort_flag && my_n < a.N) {
    const float* recv = reinterpret_cast<const float*>(smem + C::OFF_RECV);
    const int nl = static_cast<int>(threadIdx.x) % per;
    for (int m = static_cast<int>(threadIdx.x) / per; m < M; m += THREADS / per) {
      float acc = 0.f;
      for (int s = 0; s < a.splits; ++s) acc += recv[(s * NTOK + m) * per + nl];
      out[static_cast<int64_t>(m) * a.N + my_n] = __float2bfloat16_rn(fmaf(acc, alpha, bias_n));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

void fill_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int grid, int splits, int smem, cudaStream_t s) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg->blockDim = dim3(THREADS, 1, 1);
  cfg->dynamicSmemBytes = static_cast<size_t>(smem);
  cfg->stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

// Clusters of S CTAs that fit on the GPU at once, per device (asked once).
template <int FMT, int NTOK, bool kQuant>
int max_clusters(int splits, int sms) {
  static int cache[64][4] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  const int slot = splits == 8 ? 3 : (splits == 4 ? 2 : (splits == 2 ? 1 : 0));
  if (dev < 0 || dev >= 64) return sms / splits;
  if (cache[dev][slot] == 0) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    fill_config(&cfg, attr, splits, splits, Cfg<FMT, NTOK, false>::SMEM, nullptr);
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, gemm_fp4_small_kernel<FMT, NTOK, kQuant, false>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();  // the query's own error
      n = sms / splits;
    }
    cache[dev][slot] = n;
  }
  return cache[dev][slot];
}

template <int FMT, int NTOK, bool kQuant, bool kTwo>
cudaError_t launch_t(const Fp4Problem& p, int sms, cudaStream_t stream, const char** msg) {
  using C = Cfg<FMT, NTOK, kTwo>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaError_t e =
        cudaFuncSetAttribute(gemm_fp4_small_kernel<FMT, NTOK, kQuant, kTwo>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) {
      *msg = "cudaFuncSetAttribute(max dynamic shared memory) failed";
      return e;
    }
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int64_t kb = p.K / 2, RTW = ceil_div(p.N, kAtomRows), RTX = ceil_div(p.M, kAtomRows);
  const int64_t KA = ceil_div(fp4_scale_extent(FMT, p.K), kTileK);
  const int words = kAtomBytes / 4;
  CUtensorMap mw, mx, msw, msx;
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B, flat = CU_TENSOR_MAP_SWIZZLE_NONE;
  const auto l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  if (!encode_map3(&mw, u8, p.w, kb, p.N, p.B, kb, p.N * kb, BKB, ROWS, sw, l2) ||
      !encode_map3(&msw, u32, p.sfw, RTW * words, KA, p.B, RTW * kAtomBytes, KA * RTW * kAtomBytes, words, C::ATOMS,
                   flat, l2) ||
      (!kQuant &&
       (!encode_map3(&mx, u8, p.x, kb, p.M, p.B, kb, p.M * kb, BKB, NTOK, sw, l2) ||
        !encode_map3(&msx, u32, p.sfx, RTX * words, KA, p.B, RTX * kAtomBytes, KA * RTX * kAtomBytes, words, C::ATOMS,
                     flat, l2)))) {
    *msg = "cuTensorMapEncodeTiled rejected a 4-bit operand";
    return cudaErrorInvalidValue;
  }
  if (kQuant) {  // not used
    mx = mw;
    msx = msw;
  }
  Args a;
  a.x = static_cast<const __nv_bfloat16*>(p.x_bf16);
  a.K = static_cast<int>(p.K);
  a.bias = static_cast<const __nv_bfloat16*>(p.bias);
  a.gx = p.gx;
  a.gw = p.gw;
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.M = static_cast<int>(p.M);
  a.N = static_cast<int>(p.N);
  a.RTW = static_cast<int>(RTW);
  a.TT = static_cast<int>(ceil_div(p.M, NTOK));
  a.KT = static_cast<int>(ceil_div(p.K, BK));
  a.last_steps = static_cast<int>(ceil_div(p.K - static_cast<int64_t>(a.KT - 1) * BK, MMA_K));
  const int64_t tiles = p.B * a.TT * RTW;
  a.splits = 1;
  if (!kTwo) {  // the largest K split whose clusters all run at once
    a.splits = 8;
    while (a.splits > 1 && (a.splits > a.KT || tiles > max_clusters<FMT, NTOK, kQuant>(a.splits, sms))) a.splits >>= 1;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  fill_config(&cfg, attr, static_cast<int>(tiles) * a.splits, a.splits, C::SMEM, stream);
  cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_fp4_small_kernel<FMT, NTOK, kQuant, kTwo>, mw, mx, msw, msx, a);
  if (e != cudaSuccess) *msg = "small-M 4-bit GEMM launch failed";
  return e;
}

// More tiles than SMs: two CTAs an SM, each with half the ring, so that the
// tiles past the first wave stream from the start and their chains overlap
// instead of following.  Measured (us, one / two, weights from HBM): N = 28672, K
// = 4096, M = 1 15.4 / 11.5, 32 17.2 / 12.4; N = 20480, K = 5120, M = 16 17.4 /
// 11.8.  Where the tiles fit one wave the K split makes up for it: N = 14336, K =
// 4096, M = 16 8.4 with one, 8.8 with two and twice the split.
template <int FMT, int NTOK, bool kQuant>
cudaError_t launch_n(const Fp4Problem& p, int sms, cudaStream_t stream, const char** msg) {
  return p.B * ceil_div(p.M, NTOK) * ceil_div(p.N, ROWS) > sms
             ? launch_t<FMT, NTOK, kQuant, true>(p, sms, stream, msg)
             : launch_t<FMT, NTOK, kQuant, false>(p, sms, stream, msg);
}

template <int FMT>
cudaError_t launch_fmt(const Fp4Problem& p, int sms, cudaStream_t stream, const char** msg) {
  if (p.x_bf16 != nullptr) return launch_n<FMT, 16, true>(p, sms, stream, msg);
  if (p.M <= 16) return launch_n<FMT, 16, false>(p, sms, stream, msg);
  if (p.M <= 32) return launch_n<FMT, 32, false>(p, sms, stream, msg);
  if (p.M <= 64) return launch_n<FMT, 64, false>(p, sms, stream, msg);
  return launch_n<FMT, 128, false>(p, sms, stream, msg);
}

}  // namespace

namespace {

// The K split the launcher comes to on this GPU's 152 SMs, by the tile count.
int64_t splits_estimate(int64_t tiles) { return tiles <= 14 ? 8 : (tiles <= 36 ? 4 : (tiles <= 75 ? 2 : 1)); }

}  // namespace

// Quantising inside repeats the work in every CTA of the same K range, and
// saves a launch and the workspace (5 us of host time).  Measured in a graph, the
// weights from HBM (us, quantise call first / inside, MXFP4; NVFP4): N = K = 4096,
// M = 1 4.4 / 4.1, 6 4.4 / 4.4, 8 4.6 / 4.6, 16 4.7 / 5.5; 4.7 / 4.2, 4.7 / 4.8, 4.8
// / 5.3, 5.0 / 6.4; N = 14336, K = 4096, M = 1 7.8 / 7.4, 8 8.1 / 8.3, 16 8.5 / 9.7;
// N = 28672, K = 4096, M = 8 12.3 / 11.2; 12.8 / 12.1; N = 4096, K = 14336, M = 8
// 8.9 / 8.6; 9.5 / 9.4, 16 9.1 / 9.8; 9.8 / 12.1.  So in a graph NVFP4 is up to
// 10 % the slower one from six tokens on; in eager calls the host's time decides.
bool fp4_quantizes_inside(int64_t B, int64_t M) { return B == 1 && M <= QUANT_MAX_M; }

// Where this kernel is the faster one (a function of the shape alone: the
// workspace size depends on it).  Up to 64 tokens always, while two CTAs an SM
// hold the tiles; above, by its time: 0.26 us a stage of a CTA's K range, and the
// rest by the split and the tokens, which share the epilogue out but add an
// exchange.  Measured (us, MXFP4, this kernel / CTA pairs): N = K = 4096, M = 64
// 5.4 / 8.1, 128 7.3 / 8.2, 256 10.5 / 8.1, 512 9.8 / 8.5; N = K = 8192, M = 64 9.8
// / 11.0, 128 12.8 / 11.1; N = K = 2048, M = 96 5.4 / 6.2, 256 6.7 / 6.1, 512 9.5 /
// 6.2; N = 14336, K = 4096, M = 64 8.1 / 8.9, 128 9.8 / 9.2; N = 4096, K = 14336, M
// = 128 9.9 / 12.1, 256 16.1 / 13.5; 16 x [M, 512, 7168], M = 64 9.4 / 10.3, 128
// 12.3 / 10.5.  Two CTAs an SM, weights from HBM: N = 28672, K = 4096, M = 16 11.7
// / 18.7, 64 13.4 / 18.0, 128 16.2 / 18.6, 192 (448 tiles) 26.8 / 18.9; N = 32000,
// K = 2048, M = 128 11.8 / 12.9; N = 14336, K = 4096, M = 192 (224 tiles of two
// token tiles) 13.9 / 11.9; N = 128256, K = 4096 (1002 tiles), M = 32 50.9 / 60.1,
// 64 56.4 / 52.6.
bool fp4_use_small(int64_t B, int64_t M, int64_t N, int64_t K) {
  if (M <= 32) return true;
  const int64_t tiles = B * ceil_div(M, 128) * ceil_div(N, ROWS);
  if (tiles > 152) return M <= 128 && tiles <= 304;  // two CTAs an SM, all at once
  if (M <= 64) return true;
  const int64_t splits = splits_estimate(tiles), more = (M < 128 ? M : 128) - 64;
  const int64_t fixed = splits == 1 ? 375 + 3 * more
                                    : (splits == 2 ? 510 + 5 * more : (splits == 4 ? 420 : 350) + 3 * more);
  return fixed + 26 * ceil_div(ceil_div(K, BK), splits) <= fp4_pair_cost(B, M, N, K);  // 0.01 us
}

cudaError_t launch_gemm_fp4_small(const Fp4Problem& p, int sms, cudaStream_t stream, const char** msg) {
  return p.fmt == kQNV4 ? launch_fmt<kQNV4>(p, sms, stream, msg) : launch_fmt<kQMX4>(p, sms, stream, msg);
}

cudaError_t take_status_fp4_small(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(unsigned int));
}

}  // namespace mx
